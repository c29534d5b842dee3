"""Refusals of the exact-attention entry points, and what they check on the
host: nothing here needs a GPU (every refused call returns before any launch)."""
import ctypes

import pytest

nys = pytest.importorskip("streaming_nystr_landmark_gb300.nys")

GOOD = dict(heads=16, kv_heads=8, d=128, dv=128, dtype=nys.NYS_BF16, scale=0.0)
A = 1 << 20   # an address that is aligned and never read


def cfg(**kw):
    g = dict(GOOD, **kw)
    return nys.NysAttnConfig(g["heads"], g["kv_heads"], g["d"], g["dv"], g["dtype"], g["scale"])


def rows(p=A, r=2048, h=128):
    return nys.NysRows(p, r, h)


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), nys.NYS_E_INVAL), (dict(kv_heads=0), nys.NYS_E_INVAL),
    (dict(heads=15), nys.NYS_E_INVAL), (dict(d=0), nys.NYS_E_INVAL),
    (dict(d=126), nys.NYS_E_INVAL), (dict(dv=2), nys.NYS_E_INVAL),
    (dict(dtype=3), nys.NYS_E_INVAL), (dict(dtype=-1), nys.NYS_E_INVAL),
    (dict(scale=-1.0), nys.NYS_E_INVAL), (dict(scale=float("nan")), nys.NYS_E_INVAL),
    (dict(scale=float("inf")), nys.NYS_E_INVAL), (dict(d=260), nys.NYS_E_UNSUPPORTED),
    (dict(dv=260), nys.NYS_E_UNSUPPORTED), (dict(heads=520), nys.NYS_E_UNSUPPORTED),
])
def test_bad_geometry(kw, code):
    with pytest.raises(nys.NysError) as e:
        nys.nys_attn_workspace_bytes(cfg(**kw), 1, 1)
    assert e.value.code == code
    lib = nys._lib
    assert lib.nys_attn_prompt(cfg(**kw), 1, 4, 4, A, None, rows(), rows(), rows(), rows(),
                               None, None, 0, None, None) == code
    pool = nys.NysPool(A, A, 4, 16)
    assert lib.nys_attn_shared(cfg(**kw), 1, pool, None, 0, A, A, 4, rows(), rows(), None,
                               None, 0, None, None) == code
    assert lib.nys_kv_write(cfg(**kw), pool, 1, rows(), rows(), A, None) == code


def test_workspace_sizes():
    c = cfg()
    assert nys.nys_attn_workspace_bytes(c, 0, 0) >= 0
    for n, r, k in ((-1, 0, 0), (0, -1, 0), (1 << 31, 1, 1), (1, 1 << 31, 1), (1, 1, -1),
                    (1, 1, 1 << 31)):
        with pytest.raises(nys.NysError):
            nys.nys_attn_workspace_bytes(c, n, r, k)
    assert nys._lib.nys_attn_workspace_bytes(c, 1, 1, 1, None) == nys.NYS_E_INVAL
    assert nys._lib.nys_attn_workspace_bytes(None, 1, 1, 1, None) == nys.NYS_E_INVAL


def _prompt(**kw):
    a = dict(cfg=cfg(), n=1, qr=4, kr=4, qo=A, ko=None, q=rows(), k=rows(), v=rows(),
             o=rows(), lse=None, ws=None, wb=0, st=None)
    a.update(kw)
    return nys._lib.nys_attn_prompt(a["cfg"], a["n"], a["qr"], a["kr"], a["qo"], a["ko"], a["q"],
                                    a["k"], a["v"], a["o"], a["lse"], a["ws"], a["wb"], a["st"],
                                    None)


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=None), nys.NYS_E_INVAL), (dict(n=-1), nys.NYS_E_INVAL),
    (dict(qr=-1), nys.NYS_E_INVAL), (dict(kr=5), nys.NYS_E_INVAL),   # k_off NULL: one length
    (dict(qo=None), nys.NYS_E_INVAL), (dict(q=None), nys.NYS_E_INVAL),
    (dict(k=rows(p=None)), nys.NYS_E_INVAL), (dict(v=rows(r=-1)), nys.NYS_E_INVAL),
    (dict(o=rows(h=-128)), nys.NYS_E_INVAL), (dict(q=rows(p=A + 1)), nys.NYS_E_ALIGN),
    (dict(lse=A + 2), nys.NYS_E_ALIGN), (dict(qo=A + 1), nys.NYS_E_ALIGN),
    (dict(ws=A + 16, wb=64), nys.NYS_E_ALIGN), (dict(st=A + 1), nys.NYS_E_ALIGN),
    (dict(k=rows(r=1 << 50)), nys.NYS_E_INVAL),
    (dict(n=0), nys.NYS_OK), (dict(qr=0, kr=0), nys.NYS_OK),
])
def test_prompt_refusals(kw, code):
    assert _prompt(**kw) == code


def _shared(**kw):
    a = dict(cfg=cfg(), n=2, pool=nys.NysPool(A, A, 4, 16), pp=A, pl=20, lens=A, table=A, w=2,
             q=rows(), o=rows(), lse=None, ws=A, wb=1 << 40, st=None)
    a.update(kw)
    return nys._lib.nys_attn_shared(a["cfg"], a["n"], a["pool"], a["pp"], a["pl"], a["lens"],
                                    a["table"], a["w"], a["q"], a["o"], a["lse"], a["ws"],
                                    a["wb"], a["st"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=None), nys.NYS_E_INVAL), (dict(n=-1), nys.NYS_E_INVAL),
    (dict(pl=-1), nys.NYS_E_INVAL), (dict(w=-1), nys.NYS_E_INVAL),
    (dict(pool=None), nys.NYS_E_INVAL), (dict(pool=nys.NysPool(None, A, 4, 16)), nys.NYS_E_INVAL),
    (dict(pool=nys.NysPool(A, A, 4, 0)), nys.NYS_E_INVAL),
    (dict(pool=nys.NysPool(A, A, -4, 16)), nys.NYS_E_INVAL),
    (dict(pool=nys.NysPool(A + 1, A, 4, 16)), nys.NYS_E_ALIGN),
    (dict(pp=None), nys.NYS_E_INVAL), (dict(lens=None), nys.NYS_E_INVAL),
    (dict(table=None), nys.NYS_E_INVAL), (dict(q=None), nys.NYS_E_INVAL),
    (dict(o=rows(p=None)), nys.NYS_E_INVAL), (dict(lens=A + 2), nys.NYS_E_ALIGN),
    (dict(ws=A + 8), nys.NYS_E_ALIGN), (dict(w=1 << 30), nys.NYS_E_UNSUPPORTED),
    (dict(n=0), nys.NYS_OK),
])
def test_shared_refusals(kw, code):
    assert _shared(**kw) == code


def test_shared_workspace_too_small():
    need = nys.nys_attn_workspace_bytes(cfg(), 2, 2, 20)
    if need:
        assert _shared(ws=None, wb=0) == nys.NYS_E_BUF
        assert _shared(wb=need - 1) == nys.NYS_E_BUF


def _plan(**kw):
    a = dict(n=2, page=16, cached=A, fresh=A, free=A, nf=4, table=A, w=4, total=3, qo=A, lens=A,
             slots=A, pos=A, taken=A, st=None)
    a.update(kw)
    return nys._lib.nys_kv_plan(a["n"], a["page"], a["cached"], a["fresh"], a["free"], a["nf"],
                                a["table"], a["w"], a["total"], a["qo"], a["lens"], a["slots"],
                                a["pos"], a["taken"], a["st"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), nys.NYS_E_INVAL), (dict(page=0), nys.NYS_E_INVAL),
    (dict(cached=None), nys.NYS_E_INVAL), (dict(fresh=None), nys.NYS_E_INVAL),
    (dict(free=None), nys.NYS_E_INVAL), (dict(table=None), nys.NYS_E_INVAL),
    (dict(total=-1), nys.NYS_E_INVAL), (dict(total=1 << 31), nys.NYS_E_INVAL),
    (dict(qo=None), nys.NYS_E_INVAL), (dict(lens=None), nys.NYS_E_INVAL),
    (dict(slots=None), nys.NYS_E_INVAL), (dict(pos=None), nys.NYS_E_INVAL),
    (dict(taken=None), nys.NYS_E_INVAL), (dict(slots=A + 4), nys.NYS_E_ALIGN),
    (dict(cached=A + 1), nys.NYS_E_ALIGN), (dict(w=-1), nys.NYS_E_INVAL),
])
def test_plan_refusals(kw, code):
    assert _plan(**kw) == code


def _apart(**kw):
    """Plan arguments that do not overlap, a megabyte apart, but for those given."""
    names = ("cached", "fresh", "free", "table", "qo", "lens", "slots", "pos", "taken", "st")
    a = {x: A + (i << 20) for i, x in enumerate(names)}
    return dict(a, **kw)


@pytest.mark.parametrize("kw", [
    dict(fresh=A + (5 << 20)),              # fresh = lens
    dict(lens=A + 4),                       # lens one request into cached
    dict(qo=A), dict(free=A + (3 << 20) + 28), dict(table=A + (1 << 20) - 28),
    dict(slots=A + (7 << 20) - 8), dict(taken=A + (4 << 20) + 8), dict(st=A + (2 << 20)),
])
def test_plan_refuses_outputs_that_overlap(kw):
    """Every CTA reads all lengths while others write."""
    assert _plan(**_apart(**kw)) == nys.NYS_E_INVAL


@pytest.mark.parametrize("kw,code", [
    (dict(pool=None), nys.NYS_E_INVAL), (dict(tokens=-1), nys.NYS_E_INVAL),
    (dict(k=None), nys.NYS_E_INVAL), (dict(v=rows(p=None)), nys.NYS_E_INVAL),
    (dict(slots=None), nys.NYS_E_INVAL), (dict(slots=A + 4), nys.NYS_E_ALIGN),
    (dict(k=rows(p=A + 1)), nys.NYS_E_ALIGN), (dict(tokens=0), nys.NYS_OK),
    (dict(pool=nys.NysPool(None, None, 0, 16)), nys.NYS_OK),
])
def test_write_refusals(kw, code):
    a = dict(cfg=cfg(), pool=nys.NysPool(A, A, 4, 16), tokens=2, k=rows(), v=rows(), slots=A)
    a.update(kw)
    assert nys._lib.nys_kv_write(a["cfg"], a["pool"], a["tokens"], a["k"], a["v"], a["slots"],
                                 None) == code


def test_tensor_checks_of_the_wrapper():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        nys._dtype_code(torch.float64)
    with pytest.raises(ValueError):   # not a CUDA tensor
        nys._rows(torch.zeros(2, 4, 8), torch.float32, 4, 8, "q")
    with pytest.raises(ValueError):
        nys._ints(torch.zeros(2, dtype=torch.int32), torch.int32, (2,), "lens")


def test_error_names_the_call():
    with pytest.raises(nys.NysError, match="nys_kv_plan"):
        nys.nys_kv_plan(-1, 16, A, A, A, 1, A, 1, 1, A, A, A, A, A)


class _Tensor:
    """Stands for a CUDA tensor on a device that need not be there."""

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index, self.is_cuda = shape, dtype, index, True

    def stride(self):
        out, step = [], 1
        for n in reversed(self.shape):
            out.insert(0, step)
            step *= n
        return out

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


class _Device:
    """Stands for torch on a machine with two GPUs: notes which one is current."""

    def __init__(self, monkeypatch):
        import torch
        self.now, self.calls = 0, []
        outer = self

        class device:
            def __init__(self, index):
                self.index = index

            def __enter__(self):
                self.was, outer.now = outer.now, self.index

            def __exit__(self, *a):
                outer.now = self.was

        class cuda:
            @staticmethod
            def is_current_stream_capturing():
                return False
        cuda.device = device
        self.cuda = cuda
        for name in ("int32", "int64", "float32", "uint8"):
            setattr(self, name, getattr(torch, name))
        self.empty = lambda n, dtype, device: _Tensor((n,), dtype, device.index)
        self._C = type("_C", (), dict(_cuda_getDevice=lambda: self.now,
                                      _cuda_getCurrentRawStream=lambda index: 1000 + index))
        for name in ("nys_attn_prompt", "nys_attn_shared", "nys_kv_plan", "nys_kv_write"):
            monkeypatch.setattr(nys, name, lambda *a, name=name: self.calls.append(
                (name, self.now, a[-1])))


def _objects(monkeypatch, index):
    torch = pytest.importorskip("torch")
    fake, dev = _Device(monkeypatch), torch.device("cuda", index)
    att = nys.ExactAttention.__new__(nys.ExactAttention)
    vars(att).update(torch=fake, device=dev, dtype=torch.float32, heads=2, kv_heads=2, d=8, dv=8,
                     cfg=nys.NysAttnConfig(2, 2, 8, 8, nys.NYS_F32, 0.0), _work=None,
                     _work_ptr=None, _work_bytes=0, _sizes=None, _captured=False, _held=[],
                     _status_ptr=A)
    cache = nys.PagedKV.__new__(nys.PagedKV)
    vars(cache).update(torch=fake, device=dev, dtype=torch.float32, kv_heads=2, d=8, dv=8, page=4,
                       n_pages=2, _cfg=att.cfg, _pool=nys.NysPool(A, A, 2, 4))
    plan = nys.PagePlan.__new__(nys.PagePlan)
    vars(plan).update(torch=fake, device=dev, n=3, width=2, total=3, page=4, _out=[A] * 5,
                      _status_ptr=A)
    f = lambda *s, i=index: _Tensor(s, torch.float32, i)
    i32 = lambda *s, i=index: _Tensor(s, torch.int32, i)
    i64 = lambda *s, i=index: _Tensor(s, torch.int64, i)
    calls = {
        "nys_attn_prompt": (att.prompt, [f(3, 2, 8), f(3, 2, 8), f(3, 2, 8), i32(2), f(3, 2, 8),
                                         i32(2), f(3, 2)]),
        "nys_attn_shared": (att.shared, [f(3, 2, 8), cache, i32(3), i32(3, 2), f(3, 2, 8), i32(2),
                                         5, f(3, 2)]),
        "nys_kv_plan": (plan.update, [i32(3), i32(3), i32(4), i32(3, 2)]),
        "nys_kv_write": (cache.write, [f(3, 2, 8), f(3, 2, 8), i64(3)]),
    }
    return fake, calls


@pytest.mark.parametrize("name", ["nys_attn_prompt", "nys_attn_shared", "nys_kv_plan",
                                  "nys_kv_write"])
def test_calls_run_on_their_objects_device(monkeypatch, name):
    """Whichever device is current: a legacy default stream is the current device's,
    whatever the tensors are."""
    for index in (0, 1):
        fake, calls = _objects(monkeypatch, index)
        fn, args = calls[name]
        fn(*args)
        assert fake.calls == [(name, index, 1000 + index)] and fake.now == 0


@pytest.mark.parametrize("name", ["nys_attn_prompt", "nys_attn_shared", "nys_kv_plan",
                                  "nys_kv_write"])
def test_tensors_of_another_device_are_refused(monkeypatch, name):
    fake, calls = _objects(monkeypatch, 1)
    fn, args = calls[name]
    for i, a in enumerate(args):
        if not isinstance(a, _Tensor):
            continue
        a.index = 0
        with pytest.raises(ValueError, match="cuda:0"):
            fn(*args)
        a.index = 1
    if name == "nys_attn_shared":
        import torch
        args[1].device = torch.device("cuda", 0)
        with pytest.raises(ValueError, match="cuda:0"):
            fn(*args)
    assert fake.calls == []


@pytest.mark.parametrize("role", [0, 3, -1])
def test_stall_hook_refuses_unknown_roles(role):
    assert nys._lib.nys_debug_stall_attn_once(role) == nys.NYS_E_INVAL


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf")])
def test_scale_has_to_be_positive(scale):
    """0 stands for 1/sqrt(d) in the C call: given here it was taken for that."""
    pytest.importorskip("torch")
    with pytest.raises(ValueError, match="scale"):
        nys.ExactAttention(2, 2, 8, 8, scale=scale)


def test_prefix_without_pages_is_refused(monkeypatch):
    fake, calls = _objects(monkeypatch, 0)
    fn, args = calls["nys_attn_shared"]
    args[5] = None
    with pytest.raises(ValueError, match="prefix_pages"):
        fn(*args)
    assert fake.calls == []
