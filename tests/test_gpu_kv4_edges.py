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


@pytest.mark.parametrize("geo", GEOMETRIES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_lengths_past_the_table(cuda_device, dtype, geo):
    """Taken as all that the table has room for: the bits of a call with that length."""
    torch, ref, nys = _mods()
    dt, lens = getattr(torch, dtype), [48, 2496, 16]
    cache, table, slots, q, at, att, out, lse = _made(torch, nys, cuda_device, lens, geo, dt)
    cap = table.shape[1] * 16
    assert cap == 2496
    table[0], table[2] = table[1], table[1].flip(0)   # every request has pages for that many
    want, want_lse = out.clone(), lse.clone()
    at[:] = cap
    att.paged4(q, cache, at, table, want, lse=want_lse)
    assert att.status() == 0
    for n in (cap + 1, cap + 1000, 2 ** 31 - 1):
        at[0], at[2] = n, n
        att.clear_status()
        att.paged4(q, cache, at, table, out, lse=lse)
        assert att.status() == nys.NYS_ATTN_BAD_LENGTH
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    for n in (-1, -2 ** 31):
        at[0] = n
        att.paged4(q, cache, at, table, out, lse=lse)
        assert not bool(out[0].any()) and bool((lse[0] == -math.inf).all())
        assert torch.equal(out[1:], want[1:]) and torch.equal(lse[1:], want_lse[1:])


# heads, kv_heads, d, dv: 5 to 8 heads over three and four groups, 3 to 4 over three, 1 to 2 over
# four, and each kind over one and two groups
DIGITS = [(8, 1, 256, 256), (16, 2, 192, 192), (3, 1, 192, 132), (2, 1, 256, 256), (4, 1, 256, 200),
          (2, 2, 192, 192), (8, 1, 128, 128), (8, 1, 64, 64), (16, 8, 128, 128), (4, 1, 128, 128), (1, 1, 64, 64),
          (24, 2, 96, 80)]


@pytest.mark.parametrize("geo", DIGITS)
@pytest.mark.parametrize("keys", [2, 17, 300, 2000])
def test_f32_results_keep_their_digits(cuda_device, geo, keys):
    """What kv4_digits says of a result in f32, which one piece of a weight does not reach."""
    import kv4_digits
    torch, ref, nys = _mods()
    lens = [keys] * 3
    cache, table, slots, q, at, att, out, lse = _made(torch, nys, cuda_device, lens, geo, torch.float32)
    att.paged4(q, cache, at, table, out, lse=lse)
    (kc, ks, km), (vc, vs, vm) = ref.unpack(cache.data, geo[1], geo[2], geo[3], 16)
    for i, s in enumerate(slots):
        k, v = ref.values(kc[s], ks[s], km[s]), ref.values(vc[s], vs[s], vm[s])
        want, total, _ = ref.attend(q[i], k, v, 1 / math.sqrt(geo[2]), torch.float32)
        assert kv4_digits.off(out[i].double().cpu(), want) <= kv4_digits.MOST
        assert float((lse[i].double().cpu() - total).abs().max()) <= kv4_digits.MOST * 4


@pytest.mark.parametrize("geo", DIGITS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_16_bit_results_of_all_forms(cuda_device, dtype, geo):
    from test_gpu_kv4 import _check
    torch, ref, nys = _mods()
    dt, lens = getattr(torch, dtype), [0, 1, 31, 33, 700, 2100]
    cache, table, slots, q, at, att, out, lse = _made(torch, nys, cuda_device, lens, geo, dt)
    att.paged4(q, cache, at, table, out, lse=lse)
    _check(torch, ref, cache, slots, q, out, lse, geo[0], 1 / math.sqrt(geo[2]), dt)
    assert att.status() == 0


@pytest.mark.parametrize("heads", [8, 16, 32, 64])
def test_many_keys_in_f32(cuda_device, heads):
    """Over 400,000 keys that have nothing in common the result is 1/630 of a value's size, and
    codes less 8, which are -1/2 on average, would be sums of one sign.  The matrix units cut
    every sum towards zero, by up to 2^-23 of it, half that on average: even so in at most 4
    products over 32 tokens, whose sum is 16 steps in the end and half of that on the way, that is
    2 * 2^-24 * 16 steps of 0.32 of a value's size for 32 tokens, or 0.32 * 2^-24 of it for
    one; times 630, 1.2e-5.  (Sums that go on for all of a warp's keys are off by more.)"""
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


def _shifted(torch, shape, by, more, dt, dev, g=None):
    """A [rows][heads][dim] tensor whose rows start `by` numbers into rows that are `more` longer."""
    rows, heads, dim = shape
    wide = torch.full((rows, heads, dim + more), 7.0, dtype=dt, device=dev)
    if g is not None:
        wide.copy_(torch.randn(wide.shape, generator=g, device=dev))
    return wide, wide[..., by:by + dim]


@pytest.mark.parametrize("by,more", [(1, 1), (2, 3), (3, 5)])
@pytest.mark.parametrize("geo", [(16, 8, 128, 128), (4, 1, 64, 80), (8, 1, 256, 256), (6, 3, 36, 4)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_no_alignment(cuda_device, dtype, geo, by, more):
    """Rows that start anywhere, single numbers apart, give the bits that aligned ones do: norm,
    rotation, both caches, rows read back, attention."""
    torch, ref, nys = _mods()
    dt, dev, n = getattr(torch, dtype), cuda_device, 37
    heads, kv, d, dv = geo
    g = torch.Generator(device=dev).manual_seed(31)
    make = lambda h, c, gen=None: _shifted(torch, (n, h, c), by, more, dt, dev, gen)  # noqa: E731
    (_, q), (_, k), (_, v) = make(heads, d, g), make(kv, d, g), make(kv, dv, g)
    aligned = [x.contiguous() for x in (q, k, v)]
    pos = torch.randint(0, 5000, (n,), generator=g, device=dev, dtype=torch.int32)
    slots = torch.randperm(48, generator=g, device=dev)[:n]
    for rot, inter in ((d, False), (d // 2 + 2, False), (d, True), (0, False)):
        rotation = nys.Rotation(d, rot=rot, interleaved=inter, device=dev) if rot else None
        w = [1 + 0.1 * torch.randn(d, generator=g, device=dev) for _ in range(2)]
        prep = nys.QKPrepare(heads, kv, d, dtype=dt, q_weight=w[0], k_weight=w[1], rotation=rotation, device=dev)
        want = [torch.empty_like(x) for x in aligned[:2]]
        prep.rows(aligned[0], aligned[1], pos, *want)
        (wq, qo), (wk, ko) = make(heads, d), make(kv, d)
        prep.rows(q, k, pos, qo, ko)
        for x, y, wide in ((qo, want[0], wq), (ko, want[1], wk)):
            # (A row over other lanes sums its squares in another order: each is off by this.)
            size = torch.full(y.shape, 2 * float(y.abs().max()), dtype=torch.float64, device=dev)
            near = 2 * ref.turned_bound(y.double(), size, dt)
            ref.check(x, y.double(), near, "rows")
            assert bool((wide[..., :by] == 7).all()) and bool((wide[..., by + x.shape[2]:] == 7).all())
        caches = [nys.PagedKV(3, 16, kv, d, dv, dtype=dt, device=dev),
                  nys.PagedKV4(3, 16, kv, d, dv, dtype=dt, device=dev)]
        caches[0].k.fill_(7.0)
        caches[0].v.fill_(7.0)
        (_, qo), (_, ko) = make(heads, d), make(kv, d)
        for cache in caches:
            prep.append(q, k, v, pos, slots, cache, q_out=qo, k_out=ko)
            for x, y in ((qo, want[0]), (ko, want[1])):
                size = torch.full(y.shape, 2 * float(y.abs().max()), dtype=torch.float64, device=dev)
                ref.check(x, y.double(), 2 * ref.turned_bound(y.double(), size, dt), "append")
        assert torch.equal(caches[0].k.view(-1, kv, d)[slots], ko)
        assert torch.equal(caches[0].v.view(-1, kv, dv)[slots], aligned[2])
    # Codes of rows that need nothing, and back.
    four = [nys.PagedKV4(3, 16, kv, d, dv, dtype=dt, device=dev) for _ in range(2)]
    for cache, x, y in ((four[0], k, v), (four[1], *aligned[1:])):
        cache.data.zero_()
        cache.write(x, y, slots)
    assert torch.equal(four[0].data, four[1].data)
    (wk, ko), (wv, vo) = make(kv, d), make(kv, dv)
    kr, vr = torch.empty_like(aligned[1]), torch.empty_like(aligned[2])
    four[0].read(slots, ko, vo)
    four[1].read(slots, kr, vr)
    assert torch.equal(ko, kr) and torch.equal(vo, vr)
    for wide, c in ((wk, d), (wv, dv)):
        assert bool((wide[..., :by] == 7).all()) and bool((wide[..., by + c:] == 7).all())
    # Attention: queries, results and what is joined in.
    lens = torch.tensor([48, 0, 31, 17] * 9 + [5], dtype=torch.int32, device=dev)
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32, device=dev).repeat(n, 1)
    four[0].write(aligned[1].repeat(2, 1, 1)[:48], aligned[2].repeat(2, 1, 1)[:48], torch.arange(48, device=dev))
    att = nys.ExactAttention(heads, kv, d, dv, dtype=dt, device=dev)
    (_, first), (wo, out) = make(heads, dv, g), make(heads, dv)
    first_lse = torch.randn((n, heads), generator=g, device=dev)
    a = att.paged4(aligned[0], four[0], lens, table, torch.empty((n, heads, dv), dtype=dt, device=dev),
                   first=first.contiguous(), first_lse=first_lse)
    att.paged4(q, four[0], lens, table, out, first=first, first_lse=first_lse)
    assert torch.equal(out, a)
    assert bool((wo[..., :by] == 7).all()) and bool((wo[..., by + dv:] == 7).all())
