"""Attention over the 4-bit cache where a request, a row or a scale is unusual: what the
header says comes out, by whichever way the call takes."""
import math

import pytest

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16", "float16"]
# heads, kv_heads, d, dv: 1 to 2, 3 to 4 and 5 to 8 heads a KV head, and more; 1 to 4 groups
GEOMETRIES = [(16, 8, 128, 128), (4, 1, 64, 64), (32, 4, 128, 96), (20, 2, 192, 192), (2, 1, 256, 256)]


def _mods():
    import torch
    import kv4_reference as ref
    from streaming_nystr_landmark_gb300 import nys
    return torch, ref, nys


def _made(torch, nys, dev, lens, geo, dt, scale=None, seed=3):
    from test_gpu_kv4 import _cache
    heads, kv, d, dv = geo
    g = torch.Generator(device=dev).manual_seed(seed)
    cache, table, slots = _cache(torch, nys, dev, g, lens, kv, d, dv, 16, dt)
    q = torch.randn((len(lens), heads, d), generator=g, device=dev).to(dt)
    at = torch.tensor(lens, dtype=torch.int32, device=dev)
    att = nys.ExactAttention(heads, kv, d, dv, dtype=dt, device=dev, scale=scale)
    out = torch.full((len(lens), heads, dv), 7.0, dtype=dt, device=dev)
    lse = torch.full((len(lens), heads), 7.0, device=dev)
    return cache, table, slots, q, at, att, out, lse


@pytest.mark.parametrize("heads", [8, 16, 32, 64])
def test_many_keys_in_f32(cuda_device, heads):
    """Over 400,000 keys that have nothing in common the result is 1/630 of a value's size, and
    the codes less 8, of -1/2 on average, are sums of one sign.  The matrix units cut every sum
    towards zero, by up to 2^-23 of it, half that on average: in at most 4 products over 32
    tokens, whose sum is 16 steps in the end and half of that on the way, 2 * 2^-24 * 16 steps of
    0.32 of a value's size for 32 tokens, or 0.32 * 2^-24 of it for one; times 630, 1.2e-5."""
    torch, ref, nys = _mods()
    dev, n, kv, d = cuda_device, 400000, 8, 128
    g = torch.Generator(device=dev).manual_seed(23)
    cache = nys.PagedKV4(n // 64, 64, kv, d, d, device=dev)
    every = torch.arange(n, device=dev)
    k, v = (torch.randn((n, kv, d), generator=g, device=dev) for _ in range(2))
    cache.write(k, v, every)
    cache.read(every, k, v)
    at = torch.tensor([n], dtype=torch.int32, device=dev)
    table = torch.randperm(n // 64, generator=g, device=dev).int()[None]
    q = torch.randn((1, heads, d), generator=g, device=dev)
    out = torch.empty_like(q)
    nys.ExactAttention(heads, kv, d, d, device=dev).paged4(q, cache, at, table, out)
    want = torch.empty((heads, d), dtype=torch.float64, device=dev)
    for j in range(kv):
        kj, vj = k[:, j].double(), v[:, j].double()
        for h in range(j * heads // kv, (j + 1) * heads // kv):
            want[h] = (kj @ q[0, h].double() / math.sqrt(d)).softmax(0) @ vj
    assert float((out[0].double() - want).norm() / want.norm()) <= 2.0 ** -16


@pytest.mark.parametrize("geo", GEOMETRIES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("long", [33, 2500])
def test_no_keys_whatever_the_query(cuda_device, dtype, geo, long):
    """Places of a batch that hold no request: their query rows may be anything."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    lens = [0, long, 0, 17, 0]
    cache, table, slots, q, at, att, out, lse = _made(torch, nys, cuda_device, lens, geo, dt)
    clean = att.paged4(q, cache, at, table, out.clone())
    q[0], q[2, -1], q[4, :, 1] = math.nan, math.inf, -math.inf
    att.paged4(q, cache, at, table, out, lse=lse)
    for i in (0, 2, 4):
        assert not bool(out[i].any()) and bool((lse[i] == -math.inf).all())
    for i in (1, 3):
        assert torch.equal(out[i], clean[i]) and bool(lse[i].isfinite().all())
    first, first_lse = torch.randn_like(out), torch.randn_like(lse)
    att.paged4(q, cache, at, table, out, first=first, first_lse=first_lse, lse=lse)
    for i in (0, 2, 4):
        # By a factor of 1 and, for the log-sum, to base 2 and back: two roundings and two functions.
        assert torch.equal(out[i], first[i])
        assert bool(((lse[i] - first_lse[i]).abs() <= 8 * ref.U * first_lse[i].abs()).all())


@pytest.mark.parametrize("geo", GEOMETRIES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1e-8, 1e-30, 1e-44])
def test_small_scales(cuda_device, dtype, geo, scale):
    """Scores that a scale or a query row of zeros makes small leave the values' mean, in
    requests that end inside a pair of blocks too."""
    from test_gpu_kv4 import _check
    torch, ref, nys = _mods()
    dt, lens = getattr(torch, dtype), [40, 33, 5, 2500]
    cache, table, slots, q, at, att, out, lse = _made(torch, nys, cuda_device, lens, geo, dt, scale)
    q[0] = 0
    q[1] *= 1e-4
    q[2, 0] = 0
    att.paged4(q, cache, at, table, out, lse=lse)
    _check(torch, ref, cache, slots, q, out, lse, geo[0], scale, dt)


@pytest.mark.parametrize("geo", GEOMETRIES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_first_result_that_is_nan(cuda_device, dtype, geo):
    """NaN in the log-sum of what is joined in reaches the result, of a request without keys too."""
    torch, ref, nys = _mods()
    dt, lens = getattr(torch, dtype), [0, 40, 2500, 0]
    cache, table, slots, q, at, att, out, lse = _made(torch, nys, cuda_device, lens, geo, dt)
    first, first_lse = torch.randn_like(out), torch.randn_like(lse)
    first[:3, 0], first_lse[:3, 0] = math.nan, math.nan
    for o, s in ((out, lse), (first, first_lse)):      # apart, and in place
        att.paged4(q, cache, at, table, o, first=first, first_lse=first_lse, lse=s)
        assert bool(o[:3, 0].isnan().all()) and bool(s[:3, 0].isnan().all())
        assert not bool(o[:, 1:].isnan().any()) and not bool(s[:, 1:].isnan().any())
        assert not bool(o[3].isnan().any()) and not bool(s[3].isnan().any())


@pytest.mark.parametrize("geo", GEOMETRIES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_scores_below_fp32(cuda_device, dtype, geo):
    """A row whose scores are all below what fp32 holds is NaN, not a request without keys;
    beside another result whose log-sum it does hold they weigh nothing."""
    torch, ref, nys = _mods()
    dt, dev = getattr(torch, dtype), cuda_device
    lens = [1, 40, 2500, 0]
    cache, table, slots, q, at, att, out, lse = _made(torch, nys, dev, lens, geo, dt, 1.0)
    heads, kv, d, dv = geo
    k = torch.zeros((sum(lens), kv, d), dtype=dt, device=dev)
    k[..., 5] = 96.0
    v = torch.randn((sum(lens), kv, dv), device=dev).to(dt)
    cache.write(k, v, torch.cat(slots).to(dev))
    q[:] = 0
    q[..., 5] = -2.0 ** 126                       # scores of about -2^132
    att.paged4(q, cache, at, table, out, lse=lse)
    assert bool(out[:3].isnan().all()) and bool(lse[:3].isnan().all())
    assert not bool(out[3].any()) and bool((lse[3] == -math.inf).all())
    first, first_lse = torch.randn_like(out), torch.randn_like(lse)
    att.paged4(q, cache, at, table, out, first=first, first_lse=first_lse, lse=lse)
    assert torch.equal(out, first)
    assert bool(((lse - first_lse).abs() <= 8 * ref.U * first_lse.abs()).all())
