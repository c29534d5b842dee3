"""Norm and rotation of queries and keys, and appending to paged caches, against plain
forms in 64 bits; and against each other, bit for bit, where they share their steps."""
import pytest

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16", "float16"]
# heads, kv_heads, d, rot, interleaved, norm
SHAPES = [(16, 8, 128, 128, False, True), (32, 4, 128, 128, True, True), (1, 1, 64, 64, False, False),
          (14, 2, 80, 52, False, True), (3, 3, 36, 22, False, True), (5, 1, 4, 2, True, True),
          (8, 2, 256, 256, False, True), (4, 4, 192, 44, True, False), (2, 1, 60, 0, False, True),
          (6, 3, 200, 150, False, True), (2, 2, 132, 130, False, True)]


def _mods():
    import torch
    import kv4_reference as ref
    from streaming_nystr_landmark_gb300 import nys
    return torch, ref, nys


def _make(torch, nys, dev, dtype, heads, kv, d, rot, inter, norm, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    w = [1 + 0.2 * torch.randn(d, generator=g, device=dev) if norm else None for _ in range(2)]
    rotation = nys.Rotation(d, base=5e5, rot=rot, interleaved=inter, device=dev) if rot else None
    freqs = [5e5 ** (-2.0 * i / rot) for i in range(rot // 2)]
    return g, w, freqs, nys.QKPrepare(heads, kv, d, dtype=dtype, q_weight=w[0], k_weight=w[1],
                                      rotation=rotation, device=dev)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [1, 7, 700])
def test_rows(cuda_device, dtype, shape, tokens):
    torch, ref, nys = _mods()
    dt, (heads, kv, d, rot, inter, norm) = getattr(torch, dtype), shape
    g, w, freqs, prep = _make(torch, nys, cuda_device, dt, *shape)
    qkv = (3 * torch.randn((tokens, heads + 2 * kv, d), generator=g, device=cuda_device)).to(dt)
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
    pos = torch.randint(0, 100000, (tokens,), generator=g, device=cuda_device, dtype=torch.int32)
    before = qkv.clone()
    q_out, k_out = torch.empty((tokens, heads, d), dtype=dt, device=cuda_device), torch.empty(
        (tokens, kv, d), dtype=dt, device=cuda_device)
    prep.rows(q, k, pos if rot else None, q_out, k_out, shift=11)
    assert torch.equal(qkv, before)
    for x, y, wx, name in ((q, q_out, w[0], "q"), (k, k_out, w[1], "k")):
        want, size = ref.turned(x, wx, 1e-6, pos, freqs, inter, 11)
        ref.check(y, want, ref.turned_bound(want, size, dt, 100011), name)
    # In place, in the fused tensor: the same bits, the values untouched.
    got = prep.rows(q, k, pos, shift=11)
    assert got[0] is q and torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(qkv[:, heads + kv:], before[:, heads + kv:])
    # One of the two alone.
    alone = torch.empty_like(k_out)
    prep.rows(None, before[:, heads:heads + kv], pos, None, alone, shift=11)
    assert torch.equal(alone, k_out)


@pytest.mark.parametrize("pos", [0, -1, -123457, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("shift", [0, 2 ** 31 - 1, -2 ** 31])
def test_far_positions(cuda_device, pos, shift):
    torch, ref, nys = _mods()
    _, w, freqs, prep = _make(torch, nys, cuda_device, torch.float32, 2, 1, 128, 128, False, False)
    x = torch.randn((1, 2, 128), device=cuda_device, generator=torch.Generator(cuda_device).manual_seed(1))
    at = torch.tensor([pos], dtype=torch.int32, device=cuda_device)
    out = torch.empty_like(x)
    prep.rows(x, None, at, out, shift=shift)
    want, size = ref.turned(x, None, 0, at, freqs, False, shift)
    ref.check(out, want, ref.turned_bound(want, size, torch.float32, abs(pos) + abs(shift)), "far")


def test_given_frequencies_and_whole_turns(cuda_device):
    torch, ref, nys = _mods()
    freqs = [0.25, 0.0, 7.0, -1.5]
    rotation = nys.Rotation(12, rot=8, freqs=freqs, device=cuda_device)
    prep = nys.QKPrepare(1, 1, 12, rotation=rotation, device=cuda_device)
    g = torch.Generator(cuda_device).manual_seed(1)
    x = torch.randn((500, 1, 12), device=cuda_device, generator=g)
    at = torch.arange(500, dtype=torch.int32, device=cuda_device) - 250
    out = torch.empty_like(x)
    prep.rows(x, None, at, out)
    want, size = ref.turned(x, None, 0, at, freqs, False)
    # The plain form's angles are up to 1,750 here.
    ref.check(out, want, ref.turned_bound(want, size, torch.float32, 1750), "freqs")


@pytest.mark.parametrize("value", [0.0, float("inf"), float("nan"), 1e30, 1e-30])
def test_unusual_rows(cuda_device, value):
    torch, ref, nys = _mods()
    _, w, freqs, prep = _make(torch, nys, cuda_device, torch.float32, 1, 1, 64, 64, False, True)
    x = torch.ones((3, 1, 64), device=cuda_device)
    x[1] = 0.0
    x[1, 0, 5] = value
    pos = torch.tensor([1, 2, 3], dtype=torch.int32, device=cuda_device)
    out = torch.empty_like(x)
    prep.rows(x, None, pos, out)
    want, size = ref.turned(x, w[0], 1e-6, pos, freqs, False)
    rows = [0, 1, 2] if value in (0.0, 1e-30) else [0, 2]   # squares past f32 are the formula's inf
    ref.check(out[rows], want[rows], ref.turned_bound(want, size, torch.float32, 3)[rows], "rows")
    if value == 0.0:
        assert not bool(out[1].any())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [1, 5, 333])
def test_append(cuda_device, dtype, shape, tokens):
    """Into pages of the rows' own type: rows() and then write(), bit for bit."""
    torch, ref, nys = _mods()
    dt, (heads, kv, d, rot, inter, norm) = getattr(torch, dtype), shape
    g, w, freqs, prep = _make(torch, nys, cuda_device, dt, *shape)
    dv, page = 24, 8
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device).to(dt)
    q, k, v = rn(tokens, heads, d), rn(tokens, kv, d), rn(tokens, kv, dv)
    pos = torch.randint(0, 5000, (tokens,), generator=g, device=cuda_device, dtype=torch.int32)
    n_pages = tokens // page + 2
    slots = torch.randperm(n_pages * page, generator=g, device=cuda_device)[:tokens]
    slots[::3] = -1
    slots[1::5] = n_pages * page + 3
    caches = [nys.PagedKV(n_pages, page, kv, d, dv, dtype=dt, device=cuda_device) for _ in range(2)]
    for c in caches:
        c.k.fill_(7.0)
        c.v.fill_(7.0)
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    prep.rows(q, k, pos, want_q, want_k)
    caches[0].write(want_k, v, slots)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    assert prep.append(q, k, v, pos, slots, caches[1], q_out=q_out, k_out=k_out) is q_out
    assert torch.equal(q_out, want_q) and torch.equal(k_out, want_k)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    # Without queries and a copy of the keys; then queries in place.
    caches[1].k.fill_(7.0)
    prep.append(None, k, v, pos, slots, caches[1])
    assert torch.equal(caches[0].k, caches[1].k)
    assert prep.append(q, k, v, pos, slots, caches[1]) is q and torch.equal(q, want_q)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [3, 333])
def test_append4(cuda_device, dtype, shape, tokens):
    """Into 4 bits: the codes of the prepared keys in f32, bit for bit those that an f32
    cache's write() gives rows()'s f32 rows."""
    torch, ref, nys = _mods()
    dt, (heads, kv, d, rot, inter, norm) = getattr(torch, dtype), shape
    g, w, freqs, prep = _make(torch, nys, cuda_device, dt, *shape)
    dv, page = 24, 32
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device).to(dt)
    q, k, v = rn(tokens, heads, d), rn(tokens, kv, d), rn(tokens, kv, dv)
    pos = torch.randint(0, 5000, (tokens,), generator=g, device=cuda_device, dtype=torch.int32)
    n_pages = tokens // page + 2
    slots = torch.randperm(n_pages * page, generator=g, device=cuda_device)[:tokens]
    slots[::3] = -1
    a = nys.PagedKV4(n_pages, page, kv, d, dv, dtype=dt, device=cuda_device)
    b = nys.PagedKV4(n_pages, page, kv, d, dv, device=cuda_device)
    a.data.fill_(0x5a)
    b.data.fill_(0x5a)
    q_out, want_q = torch.empty_like(q), torch.empty_like(q)
    prep.append(q, k, v, pos, slots, a, q_out=q_out)
    prep.rows(q, None, pos, want_q)
    wide = nys.QKPrepare(heads, kv, d, q_weight=w[0], k_weight=w[1], rotation=prep.rotation,
                         device=cuda_device)
    k32 = torch.empty((tokens, kv, d), device=cuda_device)
    wide.rows(None, k.float(), pos, None, k32)
    b.write(k32, v.float(), slots)
    assert torch.equal(a.data, b.data) and torch.equal(q_out, want_q)


def test_refusals(cuda_device):
    torch, ref, nys = _mods()
    dev = cuda_device
    z = lambda n, h, d, dt=torch.float32: torch.zeros((n, h, d), dtype=dt, device=dev)
    i = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device=dev)
    rot = nys.Rotation(64, device=dev)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(q_weight=torch.ones(63, device=dev)),
                dict(rotation=nys.Rotation(32, device=dev))):
        with pytest.raises(ValueError):
            nys.QKPrepare(4, 2, 64, device=dev, **bad)
    for bad in (dict(rot=3), dict(rot=66), dict(rot=-2), dict(rot=4, freqs=[1.0]),
                dict(rot=2, freqs=[float("inf")])):
        with pytest.raises(ValueError):
            nys.Rotation(64, device=dev, **bad)
    prep = nys.QKPrepare(4, 2, 64, rotation=rot, device=dev)
    q, k, v = z(3, 4, 64), z(3, 2, 64), z(3, 2, 64)
    for call in (lambda: prep.rows(None, None, i(3)), lambda: prep.rows(q, z(2, 2, 64), i(3)),
                 lambda: prep.rows(q, k, None), lambda: prep.rows(q, k, i(2)),
                 lambda: prep.rows(q, k, i(3), shift=2 ** 31), lambda: prep.rows(q.half(), k, i(3)),
                 lambda: prep.rows(q, None, i(3), None, k), lambda: prep.rows(q, k, i(3), z(2, 4, 64)),
                 lambda: prep.rows(q[..., ::2], k, i(3)), lambda: prep.rows(q.cpu(), k, i(3))):
        with pytest.raises(ValueError):
            call()
    cache = nys.PagedKV(2, 8, 2, 64, 64, device=dev)
    s = i(3, torch.int64)
    for call in (lambda: prep.append(q, k, z(2, 2, 64), i(3), s, cache),
                 lambda: prep.append(q, k, z(3, 2, 32), i(3), s, cache),
                 lambda: prep.append(q, k, v, i(3), i(3), cache),
                 lambda: prep.append(None, k, v, i(3), s, cache, q_out=q),
                 lambda: prep.append(q, k, v, i(3), s, nys.PagedKV(2, 8, 1, 64, 64, device=dev)),
                 lambda: prep.append(q, k, v, i(3), s,
                                     nys.PagedKV(2, 8, 2, 64, 64, dtype=torch.float16, device=dev))):
        with pytest.raises(ValueError):
            call()


def test_capture_and_another_stream(cuda_device):
    torch, ref, nys = _mods()
    g, w, freqs, prep = _make(torch, nys, cuda_device, torch.bfloat16, 16, 8, 128, 128, False, True)
    cache = nys.PagedKV4(8, 16, 8, 128, 128, dtype=torch.bfloat16, device=cuda_device)
    rn = lambda h: torch.randn((5, h, 128), generator=g, device=cuda_device).bfloat16()
    q, k, v, out = rn(16), rn(8), rn(8), torch.empty_like(rn(16))
    pos = torch.arange(5, dtype=torch.int32, device=cuda_device)
    slots = torch.arange(5, device=cuda_device) + 14
    cache.data.zero_()
    prep.append(q, k, v, pos, slots, cache, q_out=out)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        prep.append(q, k, v, pos, slots, cache, q_out=out)
    for shift in (0, 3):
        pos.add_(shift)
        q.copy_(rn(16))
        k.copy_(rn(8))
        graph.replay()
        got = cache.data.clone(), out.clone()
        cache.data.zero_()
        prep.append(q, k, v, pos, slots, cache, q_out=out)
        assert torch.equal(got[0], cache.data) and torch.equal(got[1], out)
