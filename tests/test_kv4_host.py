"""Refusals of the entry points for prepared rows and the 4-bit cache, and their host
arithmetic: nothing here needs a GPU (every refused call returns before any launch)."""
import ctypes
import math

import pytest

nys = pytest.importorskip("streaming_nystr_landmark_gb300.nys")

A = 1 << 20   # an address that is aligned and never read
GOOD = dict(heads=16, kv_heads=8, d=128, dv=128, dtype=nys.NYS_BF16, scale=0.0)
E, U, AL, B = nys.NYS_E_INVAL, nys.NYS_E_UNSUPPORTED, nys.NYS_E_ALIGN, nys.NYS_E_BUF


def cfg(**kw):
    g = dict(GOOD, **kw)
    return nys.NysAttnConfig(g["heads"], g["kv_heads"], g["d"], g["dv"], g["dtype"], g["scale"])


def rows(p=A, r=2048, h=128):
    return nys.NysRows(p, r, h)


def prep(qw=A, kw=A, eps=1e-6, turns=A, rot=128, inter=0, shift=0):
    return nys.NysQkPrepare(qw, kw, eps, turns, rot, inter, shift)


BAD_CFG = [(dict(heads=0), E), (dict(heads=15), E), (dict(d=126), E), (dict(dv=0), E), (dict(dtype=3), E),
           (dict(scale=-1.0), E), (dict(d=260), U), (dict(heads=520), U)]
BAD_PREP = [(dict(eps=-1.0), E), (dict(eps=math.nan), E), (dict(eps=math.inf), E), (dict(rot=-2), E),
            (dict(rot=3), E), (dict(rot=130), E), (dict(turns=None), E), (dict(inter=2), E), (dict(qw=A + 2), AL),
            (dict(kw=A + 1), AL), (dict(turns=A + 4), AL)]


def _rows_call(**kw):
    a = dict(cfg=cfg(), prep=prep(), n=2, q=rows(), k=rows(), pos=A, qo=rows(), ko=rows())
    a.update(kw)
    return nys._lib.nys_qk_rows(a["cfg"], a["prep"], a["n"], a["q"], a["k"], a["pos"], a["qo"], a["ko"], None)


def _append(four, **kw):
    a = dict(cfg=cfg(), prep=prep(), n=2, q=rows(), k=rows(), v=rows(), pos=A, slots=A, qo=rows(), ko=rows(),
             pool=nys.NysPool4(A, 4, 16) if four else nys.NysPool(A, A, 4, 16))
    a.update(kw)
    f = nys._lib.nys_kv4_append if four else nys._lib.nys_kv_append
    return f(a["cfg"], a["prep"], a["pool"], a["n"], a["q"], a["k"], a["v"], a["pos"], a["slots"], a["qo"], a["ko"],
             None)


def _write(**kw):
    a = dict(cfg=cfg(), n=2, k=rows(), v=rows(), slots=A, pool=nys.NysPool4(A, 4, 16))
    a.update(kw)
    return nys._lib.nys_kv4_write(a["cfg"], a["pool"], a["n"], a["k"], a["v"], a["slots"], None)


def _read(**kw):
    a = dict(cfg=cfg(), n=2, k=rows(), v=rows(), slots=A, pool=nys.NysPool4(A, 4, 16))
    a.update(kw)
    return nys._lib.nys_kv4_read(a["cfg"], a["pool"], a["n"], a["slots"], a["k"], a["v"], None)


def _attn(**kw):
    a = dict(cfg=cfg(), n=2, pool=nys.NysPool4(A, 4, 16), lens=A, table=A, w=400, q=rows(), f=None, fl=None, o=rows(),
             lse=None, ws=A, wb=1 << 40, st=None)
    a.update(kw)
    return nys._lib.nys_attn4(a["cfg"], a["n"], a["pool"], a["lens"], a["table"], a["w"], a["q"], a["f"], a["fl"],
                              a["o"], a["lse"], a["ws"], a["wb"], a["st"], None)


@pytest.mark.parametrize("kw,code", BAD_CFG)
def test_bad_geometry(kw, code):
    c = cfg(**kw)
    assert _rows_call(cfg=c) == _append(False, cfg=c) == _append(True, cfg=c) == code
    assert _write(cfg=c) == _read(cfg=c) == _attn(cfg=c) == code
    out = ctypes.c_size_t(0)
    assert nys._lib.nys_kv4_page_bytes(c, 16, out) == nys._lib.nys_attn4_workspace_bytes(c, 1, 1, out) == code


@pytest.mark.parametrize("kw,code", BAD_PREP)
def test_bad_preparation(kw, code):
    p = prep(**kw)
    assert _rows_call(prep=p) == _append(False, prep=p) == _append(True, prep=p) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=None), E), (dict(prep=None), E), (dict(n=-1), E), (dict(n=1 << 31), E), (dict(pos=None), E),
    (dict(q=None, k=None, qo=None, ko=None), E), (dict(q=None), E), (dict(k=None), E), (dict(qo=None), E),
    (dict(ko=None), E), (dict(q=rows(p=None)), E), (dict(ko=rows(r=-1)), E), (dict(k=rows(r=1 << 50)), E),
    (dict(qo=rows(p=A + 1)), AL), (dict(pos=A + 2), AL), (dict(n=0), 0), (dict(n=0, pos=None), 0),
])
def test_rows_refusals(kw, code):
    assert _rows_call(**kw) == code


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), E), (dict(k=None), E), (dict(v=None), E), (dict(q=None), E), (dict(qo=None), E),
    (dict(slots=None), E), (dict(slots=A + 4), AL), (dict(pool=None), E), (dict(v=rows(h=-1)), E),
    (dict(n=0, slots=None, pos=None), 0),
])
def test_append_refusals(four, kw, code):
    assert _append(four, **kw) == code


BAD_POOL4 = [(None, E), (nys.NysPool4(None, 4, 16), E), (nys.NysPool4(A, -1, 16), E), (nys.NysPool4(A, 4, 0), E),
             (nys.NysPool4(A, 4, 8), E), (nys.NysPool4(A, 4, 24), E), (nys.NysPool4(A, 1 << 31, 16), U),
             (nys.NysPool4(A, 4, 1 << 21), U), (nys.NysPool4(A + 8, 4, 16), AL)]


@pytest.mark.parametrize("pool,code", BAD_POOL4)
def test_bad_pool(pool, code):
    assert _append(True, pool=pool) == _write(pool=pool) == _read(pool=pool) == _attn(pool=pool) == code


def test_pages_past_31_bits():
    c, pool = cfg(d=256, dv=256), nys.NysPool4(A, 1, 1 << 20)     # 2.4 GB
    assert _append(True, cfg=c, pool=pool) == _write(cfg=c, pool=pool) == _read(cfg=c, pool=pool) == U
    assert _attn(cfg=c, pool=pool, w=1) == U


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), E), (dict(n=1 << 31), E), (dict(k=None), E), (dict(v=None), E), (dict(k=rows(p=None)), E),
    (dict(v=rows(p=A + 1)), AL), (dict(slots=None), E), (dict(slots=A + 4), AL), (dict(n=0), 0),
])
def test_write_and_read_refusals(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), E), (dict(w=-1), E), (dict(lens=None), E), (dict(table=None), E), (dict(q=None), E),
    (dict(o=None), E), (dict(o=rows(p=None)), E), (dict(f=rows()), E), (dict(fl=A), E), (dict(f=rows(p=None), fl=A), E),
    (dict(f=rows(), fl=A + 2), AL), (dict(lse=A + 1), AL), (dict(lens=A + 2), AL), (dict(ws=A + 16), AL),
    (dict(st=A + 1), AL), (dict(w=1 << 30), U), (dict(n=1 << 30), E), (dict(n=0), 0),
])
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code


def test_workspace():
    need = nys.nys_attn4_workspace_bytes(cfg(), 2, 6400)
    assert need > 0 and nys.nys_attn4_workspace_bytes(cfg(), 2, 16) == 0
    assert nys.nys_attn4_workspace_bytes(cfg(), 0, 6400) == 0
    assert _attn(ws=None, wb=0) == _attn(wb=need - 1) == B
    for n, k in ((-1, 1), (1, -1), (1 << 31, 1), (1, 1 << 31)):
        with pytest.raises(nys.NysError):
            nys.nys_attn4_workspace_bytes(cfg(), n, k)


@pytest.mark.parametrize("d,dv,groups", [(4, 4, 1), (64, 64, 1), (68, 4, 2), (128, 128, 2), (80, 200, 4)])
def test_page_bytes(d, dv, groups):
    assert nys.nys_kv4_page_bytes(cfg(d=d, dv=dv), 48) == 8 * 3 * 1152 * groups
    for page in (0, 8, 24, -16, 1 << 20):
        with pytest.raises(nys.NysError):
            nys.nys_kv4_page_bytes(cfg(heads=128, kv_heads=128), page)


def test_turns():
    """turns[i] * position, modulo 2^64, is the angle as a fraction of a turn."""
    freqs = [1.0, 0.5, 1e-6, 7.0, -0.25, 0.0]
    rot = nys.Rotation(16, rot=12, freqs=freqs, device="cpu")
    for f, t in zip(freqs, rot.turns.tolist()):
        for pos in (1, 12345, -7):
            turn = (t * pos % 2 ** 64) / 2 ** 64
            assert abs(math.remainder(turn * 2 * math.pi - pos * f, 2 * math.pi)) < 1e-9


def _objects(monkeypatch, index):
    """This module's classes on a machine with two GPUs that need not be there."""
    torch = pytest.importorskip("torch")
    from test_attn_host import _Device, _Tensor
    fake, dev = _Device(monkeypatch), torch.device("cuda", index)
    for name in ("nys_qk_rows", "nys_kv_append", "nys_kv4_append", "nys_kv4_write", "nys_kv4_read", "nys_attn4"):
        monkeypatch.setattr(nys, name, lambda *a, name=name: fake.calls.append((name, fake.now, a[-1])))
    c = nys.NysAttnConfig(2, 2, 8, 8, nys.NYS_F32, 0.0)
    prep = nys.QKPrepare.__new__(nys.QKPrepare)
    vars(prep).update(torch=fake, device=dev, dtype=torch.float32, heads=2, kv_heads=2, d=8, cfg=c, _int32=torch.int32,
                      _prep=nys.NysQkPrepare(None, None, 1e-6, A, 8, 0, 0))
    att = nys.ExactAttention.__new__(nys.ExactAttention)
    vars(att).update(torch=fake, device=dev, dtype=torch.float32, heads=2, kv_heads=2, d=8, dv=8, cfg=c, _work=None,
                     _work_ptr=None, _work_bytes=0, _sizes=None, _captured=False, _held=[], _status_ptr=A)
    full, four = nys.PagedKV.__new__(nys.PagedKV), nys.PagedKV4.__new__(nys.PagedKV4)
    for cache, pool in ((full, nys.NysPool(A, A, 2, 16)), (four, nys.NysPool4(A, 2, 16))):
        vars(cache).update(torch=fake, device=dev, dtype=torch.float32, kv_heads=2, d=8, dv=8, page=16, n_pages=2,
                           _cfg=c, _pool=pool)
    f = lambda *s: _Tensor(s, torch.float32, index)
    i32 = lambda *s: _Tensor(s, torch.int32, index)
    i64 = lambda *s: _Tensor(s, torch.int64, index)
    rows = lambda: f(3, 2, 8)
    return _Tensor, fake, {
        "nys_qk_rows": (prep.rows, [rows(), rows(), i32(3), rows(), rows()]),
        "nys_kv_append": (prep.append, [rows(), rows(), rows(), i32(3), i64(3), full, rows(), rows()]),
        "nys_kv4_append": (prep.append, [rows(), rows(), rows(), i32(3), i64(3), four, rows(), rows(), 7]),
        "nys_kv4_write": (four.write, [rows(), rows(), i64(3)]),
        "nys_kv4_read": (four.read, [i64(3), rows(), rows()]),
        "nys_attn4": (att.paged4, [rows(), four, i32(3), i32(3, 2), rows(), rows(), f(3, 2), f(3, 2)]),
    }


NAMES = ["nys_qk_rows", "nys_kv_append", "nys_kv4_append", "nys_kv4_write", "nys_kv4_read", "nys_attn4"]


@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_their_objects_device(monkeypatch, name):
    for index in (0, 1):
        _, fake, calls = _objects(monkeypatch, index)
        fn, args = calls[name]
        fn(*args)
        assert fake.calls == [(name, index, 1000 + index)] and fake.now == 0


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(monkeypatch, name):
    _Tensor, fake, calls = _objects(monkeypatch, 1)
    fn, args = calls[name]
    for a in args:
        if isinstance(a, _Tensor):
            a.index = 0
            with pytest.raises(ValueError, match="cuda:0"):
                fn(*args)
            a.index = 1
        elif isinstance(a, (nys.PagedKV, nys.PagedKV4)):
            import torch
            a.device = torch.device("cuda", 0)
            with pytest.raises(ValueError, match="cuda:0"):
                fn(*args)
            a.device = torch.device("cuda", 1)
    assert fake.calls == []
