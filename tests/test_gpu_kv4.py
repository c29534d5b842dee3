"""The 4-bit paged cache and attention over it, against plain forms: codes and scales bit
for bit, attention against 64 bits over the values that the codes stand for."""
import math

import pytest

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16", "float16"]


def _mods():
    import torch
    import kv4_reference as ref
    from streaming_nystr_landmark_gb300 import nys
    return torch, ref, nys


# kv_heads, d, dv, page
GEOMETRIES = [(8, 128, 128, 16), (1, 64, 64, 48), (2, 80, 96, 32), (3, 36, 4, 16), (2, 256, 192, 64),
              (1, 132, 60, 16)]


@pytest.mark.parametrize("geo", GEOMETRIES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [1, 19, 200])
def test_write_and_read(cuda_device, dtype, geo, tokens):
    torch, ref, nys = _mods()
    dt, (kv, d, dv, page) = getattr(torch, dtype), geo
    g = torch.Generator(device=cuda_device).manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device)
    # Rows inside a wider tensor, with a mean and scales of their own.
    wide = (rn(tokens, 2 * kv, d + dv) * torch.exp(2 * rn(tokens, 2 * kv, 1)) + 2 * rn(1, 2 * kv, 1)).to(dt)
    k, v = wide[:, kv:, :d], wide[:, :kv, d:]
    n_pages = tokens // page + 2
    slots = torch.randperm(n_pages * page, generator=g, device=cuda_device)[:tokens]
    written = torch.ones(tokens, dtype=torch.bool, device=cuda_device)
    if tokens > 1:
        slots[3::7], written[3::7] = -1, False
        slots[5::11], written[5::11] = n_pages * page, False
    cache = nys.PagedKV4(n_pages, page, kv, d, dv, dtype=dt, device=cuda_device)
    assert cache.data.numel() == n_pages * kv * (page // 16) * 1152 * -(-max(d, dv) // 64)
    cache.data.random_(generator=g)
    before = ref.unpack(cache.data, kv, d, dv, page)
    cache.write(k, v, slots)
    after = ref.unpack(cache.data, kv, d, dv, page)
    mine = slots[written].cpu()
    others = torch.ones(n_pages * page, dtype=torch.bool)
    others[mine] = False
    every = torch.arange(n_pages * page, device=cuda_device)
    got = [torch.empty((n_pages * page, kv, c), dtype=dt, device=cuda_device) for c in (d, dv)]
    cache.read(every, *got)
    for x, old, new, y in zip((k, v), before, after, got):
        want = ref.quantize(x[written])
        for a, b, c in zip(want, new, old):
            assert torch.equal(a, b[mine].to(a.dtype)) and torch.equal(b[others].nan_to_num(), c[others].nan_to_num())
        held = ref.values(*(t[mine] for t in new))
        step = new[1][mine].double().repeat_interleave(64, -1)[..., :x.shape[-1]]
        # Half a step, more by the rounding of x - mid, of the quotient (at most 8) and of
        # the bounds that the step comes from.
        slack = (x[written].double().cpu().abs() + 8 * step) * 4 * ref.U
        assert bool(((held - x[written].double().cpu()).abs() <= step / 2 + slack).all())
        # read(): their sum rounded to f32, and that to the rows' type.
        assert torch.equal(y.cpu()[mine], held.float().to(dt))
    some = torch.tensor([-1, n_pages * page, int(mine[0]) if len(mine) else 0], device=cuda_device)
    few = [torch.full((3, kv, c), 7.0, dtype=dt, device=cuda_device) for c in (d, dv)]
    cache.read(some, *few)
    assert not bool(few[0][:2].any()) and not bool(few[1][:2].any())


@pytest.mark.parametrize("case", ["zeros", "equal", "nan", "inf", "both", "spread", "small", "subnormal", "ramp",
                                  "odd equal", "large"])
def test_unusual_groups(cuda_device, case):
    torch, ref, nys = _mods()
    x = torch.randn((4, 1, 128), generator=torch.Generator().manual_seed(2))
    part = x[1, 0, 64:]
    if case == "zeros":
        part.zero_()
    elif case == "equal":
        part.fill_(-3.140625)      # bf16 holds it
    elif case == "odd equal":
        part.fill_(1.2345678)
    elif case == "nan":
        part[17] = math.nan
    elif case == "inf":
        part[63] = math.inf
    elif case == "both":
        part[0], part[1] = math.inf, -math.inf
    elif case == "spread":
        part[3], part[4] = 3e38, -3e38
    elif case == "large":
        part.mul_(2.0 ** 120)
    elif case == "small":
        part.mul_(2.0 ** -110)
    elif case == "subnormal":
        part.mul_(2.0 ** -130)
    else:
        part.copy_(torch.arange(64) / 4.0)   # ties among them
    x = x.to(cuda_device)
    cache = nys.PagedKV4(1, 16, 1, 128, 128, device=cuda_device)
    cache.write(x, x.flip(0), torch.arange(4, device=cuda_device) + 7)
    new = ref.unpack(cache.data, 1, 128, 128, 16)
    for y, got in ((x, new[0]), (x.flip(0), new[1])):
        for a, b in zip(ref.quantize(y), got):
            assert torch.equal(torch.nan_to_num(a, 5.0), torch.nan_to_num(b[7:11].to(a.dtype), 5.0))
            assert torch.equal(a.isnan(), b[7:11].isnan())
    k, v = torch.empty_like(x), torch.empty_like(x)
    cache.read(torch.arange(4, device=cuda_device) + 7, k, v)
    bad = case in ("nan", "inf", "both", "spread")
    assert bool(k[1, 0, 64:].isnan().all()) == bad and not bool(k[1, 0, :64].isnan().any())
    if case in ("zeros", "equal"):
        assert torch.equal(k[1, 0, 64:], x[1, 0, 64:])


def _cache(torch, nys, dev, g, lens, kv, d, dv, page, dtype, extra=0, poison=True):
    """A cache whose requests' rows are drawn, every other byte of it NaN scales; the table
    has `extra` more columns, of numbers that are no pages."""
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + 2
    cache = nys.PagedKV4(n_pages, page, kv, d, dv, dtype=dtype, device=dev)
    cache.data.fill_(0xff if poison else 0)
    order = torch.randperm(n_pages, generator=g, device=dev).int().cpu()
    width = max(max(need), 1) + extra
    table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
    at, slots = 0, []
    for i, x in enumerate(lens):
        table[i, :need[i]] = order[at:at + need[i]]
        at += need[i]
        j = torch.arange(x)
        slots.append(table[i].long()[j // page] * page + j % page)
    rows = sum(lens)
    mean = 2 * torch.randn((1, kv, d), generator=g, device=dev) / math.sqrt(d)
    k = (torch.randn((rows, kv, d), generator=g, device=dev) + mean).to(dtype)
    v = torch.randn((rows, kv, dv), generator=g, device=dev).to(dtype)
    if rows:
        cache.write(k, v, torch.cat(slots).to(dev))
    return cache, table.to(dev), slots


def _check(torch, ref, cache, slots, q, out, lse, heads, scale, dtype, first=None, first_lse=None):
    (kc, ks, km), (vc, vs, vm) = ref.unpack(cache.data, cache.kv_heads, cache.d, cache.dv, cache.page)
    for i, s in enumerate(slots):
        k, v = ref.values(kc[s], ks[s], km[s]), ref.values(vc[s], vs[s], vm[s])
        want, total, bound = ref.attend(q[i], k, v, scale, dtype)
        if len(s):
            lb = ref.lse_bound(q[i], k, scale, total)
        else:
            lb = torch.zeros(heads, dtype=torch.float64)
        if first is not None:
            f, fl = first[i].double().cpu(), first_lse[i].double().cpu()
            both = torch.logaddexp(total, fl)
            dead = torch.isinf(both)
            wa = torch.where(dead, 0.0, torch.exp(total - torch.where(dead, 0.0, both)))
            wb = torch.where(dead, 0.0, torch.exp(fl - torch.where(dead, 0.0, both)))
            # Weights go by the log-sums: off by their errors, and by an exponential's.
            shift = (lb + 2 * ref.U * (fl.abs().nan_to_num(0, 0, 0) + 32))[:, None]
            joined = wa[:, None] * want + wb[:, None] * f
            bound = bound + 2 * shift * (want.abs() + f.abs()) + ref.EPS[dtype] * joined.abs() + 4 * ref.U * joined.abs()
            want, total = joined, both
            lb = lb + 4 * ref.U * (both.abs().nan_to_num(0, 0, 0) + 64)
        ref.check(out[i], want, bound, f"request {i} of {len(s)}")
        if lse is not None:
            dead = torch.isinf(total)
            assert torch.equal(torch.isinf(lse[i].cpu()), dead)
            ref.check(torch.where(dead, 0.0, lse[i].cpu()), torch.where(dead, 0.0, total), lb + 1e-30, f"lse {i}")


# heads, kv_heads, d, dv, page
ATTEND = [(16, 8, 128, 128, 16), (32, 4, 128, 128, 64), (1, 1, 64, 64, 16), (14, 2, 80, 80, 48),
          (9, 1, 64, 128, 16), (64, 1, 64, 64, 32), (3, 3, 36, 4, 16), (4, 2, 192, 132, 16), (8, 2, 256, 256, 32)]
LENGTHS = [[0], [1], [15, 16, 17, 0, 33], [300, 1, 128, 129, 31], [2000, 5]]


@pytest.mark.parametrize("geo", ATTEND)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENGTHS)
def test_attention(cuda_device, dtype, geo, lens):
    torch, ref, nys = _mods()
    dt, (heads, kv, d, dv, page) = getattr(torch, dtype), geo
    g = torch.Generator(device=cuda_device).manual_seed(3)
    cache, table, slots = _cache(torch, nys, cuda_device, g, lens, kv, d, dv, page, dt, extra=1)
    # Strided queries and results.
    wide = torch.randn((len(lens), heads, d + 12), generator=g, device=cuda_device).to(dt)
    q = wide[..., 4:4 + d]
    room = torch.full((len(lens), heads + 1, dv + 4), 7.0, dtype=dt, device=cuda_device)
    out = room[:, 1:, :dv]
    lse = torch.empty((len(lens), heads), device=cuda_device)
    at = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    att = nys.ExactAttention(heads, kv, d, dv, dtype=dt, device=cuda_device)
    assert att.paged4(q, cache, at, table, out, lse=lse) is out
    _check(torch, ref, cache, slots, q, out, lse, heads, 1 / math.sqrt(d), dt)
    assert bool((room[:, 0] == 7).all()) and bool((room[..., dv:] == 7).all()) and att.status() == 0
    # Again, without the log-sums, bit for bit.
    again = torch.empty((len(lens), heads, dv), dtype=dt, device=cuda_device)
    att.paged4(q, cache, at, table, again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_short_requests(cuda_device, dtype):
    """More units than warps: shares that end anywhere, in the middle of requests too."""
    torch, ref, nys = _mods()
    dt, (heads, kv, d) = getattr(torch, dtype), (16, 8, 64)
    g = torch.Generator(device=cuda_device).manual_seed(4)
    lens = [int(x) for x in torch.randint(0, 150, (611,), generator=torch.Generator().manual_seed(5))]
    lens[17], lens[300], lens[610] = 2500, 0, 1100
    cache, table, slots = _cache(torch, nys, cuda_device, g, lens, kv, d, d, 16, dt)
    q = torch.randn((len(lens), heads, d), generator=g, device=cuda_device).to(dt)
    out, lse = torch.empty_like(q), torch.empty((len(lens), heads), device=cuda_device)
    at = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    att.paged4(q, cache, at, table, out, lse=lse)
    _check(torch, ref, cache, slots, q, out, lse, heads, 1 / math.sqrt(d), dt)
    assert att.status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("place", ["apart", "in place"])
def test_joined_with_a_prefix(cuda_device, dtype, place):
    torch, ref, nys = _mods()
    dt, (heads, kv, d, dv) = getattr(torch, dtype), (8, 2, 128, 64)
    g = torch.Generator(device=cuda_device).manual_seed(6)
    lens = [0, 0, 5, 400, 1500, 16]
    cache, table, slots = _cache(torch, nys, cuda_device, g, lens, kv, d, dv, 16, dt)
    q = torch.randn((len(lens), heads, d), generator=g, device=cuda_device).to(dt)
    first = torch.randn((len(lens), heads, dv), generator=g, device=cuda_device).to(dt)
    first_lse = 4 + 3 * torch.randn((len(lens), heads), generator=g, device=cuda_device)
    first_lse[0], first_lse[3, 1] = -math.inf, -math.inf
    first[0] = math.nan                       # weight 0: never looked at
    kept, kept_lse = first.clone(), first_lse.clone()
    kept[0] = 0
    out, lse = (first, first_lse) if place == "in place" else (torch.empty_like(first), torch.empty_like(first_lse))
    at = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    att = nys.ExactAttention(heads, kv, d, dv, dtype=dt, device=cuda_device)
    att.paged4(q, cache, at, table, out, first=first, first_lse=first_lse, lse=lse)
    _check(torch, ref, cache, slots, q, out, lse, heads, 1 / math.sqrt(d), dt, kept, kept_lse)


def test_bad_pages_and_lengths(cuda_device):
    torch, ref, nys = _mods()
    heads, kv, d, page = 4, 2, 64, 16
    g = torch.Generator(device=cuda_device).manual_seed(7)
    lens = [40, 40, 40]
    cache, table, slots = _cache(torch, nys, cuda_device, g, lens, kv, d, d, page, torch.float32)
    q = torch.randn((3, heads, d), generator=g, device=cuda_device)
    out = torch.empty_like(q)
    att = nys.ExactAttention(heads, kv, d, d, device=cuda_device)
    at = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    good = att.paged4(q, cache, at, table, out).clone()
    for bad in (-1, cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 1] = bad
        att.clear_status()
        att.paged4(q, cache, at, t, out)
        assert att.status() == nys.NYS_ATTN_BAD_PAGE
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        # Its 16 keys and values count as 0.
        (kc, ks, km), (vc, vs, vm) = ref.unpack(cache.data, kv, d, d, page)
        k, v = ref.values(kc, ks, km)[slots[1]], ref.values(vc, vs, vm)[slots[1]]
        k[16:32] = 0
        v[16:32] = 0
        want, _, bound = ref.attend(q[1], k, v, 1 / math.sqrt(d), torch.float32)
        ref.check(out[1], want, bound, "bad page")
    for bad, taken in ((-5, 0), (1000, table.shape[1] * page)):
        at[2] = bad
        att.clear_status()
        if taken:
            cache.data.zero_()   # every slot holds something: zeros
            t = torch.zeros_like(table)
        else:
            t = table
        att.paged4(q, cache, at, t, out)
        assert att.status() == nys.NYS_ATTN_BAD_LENGTH
        assert not bool(out[2].any())


def test_unusual_values(cuda_device):
    """NaN in a group reaches the requests that see it and nobody else; queries of any size,
    all equal scores, scores far apart."""
    torch, ref, nys = _mods()
    heads, kv, d, page = 2, 1, 64, 16
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(8)
    lens = [50, 50, 50]
    cache, table, slots = _cache(torch, nys, dev, g, lens, kv, d, d, page, torch.float32)
    q = torch.randn((3, heads, d), generator=g, device=dev)
    att = nys.ExactAttention(heads, kv, d, d, device=dev)
    at = torch.tensor(lens, dtype=torch.int32, device=dev)
    out, lse = torch.empty_like(q), torch.empty((3, heads), device=dev)
    for size in (1e-30, 1e-4, 1.0, 30.0, 1e4):
        x = q * size
        att.paged4(x, cache, at, table, out, lse=lse)
        _check(torch, ref, cache, slots, x, out, lse, heads, 1 / math.sqrt(d), torch.float32)
    x = q.clone()
    x[0] = 0
    x[2, 1, 3] = math.inf
    att.paged4(x, cache, at, table, out, lse=lse)
    _check(torch, ref, cache, slots[:2], x, out, lse, heads, 1 / math.sqrt(d), torch.float32)
    assert bool(out[2, 1].isnan().all()) and not bool(out[2, 0].isnan().any())
    row = torch.randn((1, 1, d), generator=g, device=dev)
    row[0, 0, 9] = math.nan
    cache.write(row, row, slots[1][49:50].to(dev))
    att.paged4(q, cache, at, table, out)
    assert bool(out[1].isnan().all()) and not bool(out[0].isnan().any()) and not bool(out[2].isnan().any())
    at[1] = 49      # not seen any more
    att.paged4(q, cache, at, table, out)
    assert not bool(out.isnan().any()) and att.status() == 0


def test_empty_tables_and_pools(cuda_device):
    """No columns, no pages, no requests: zeros, or what is joined in."""
    torch, ref, nys = _mods()
    dev = cuda_device
    att = nys.ExactAttention(4, 2, 64, 64, device=dev)
    q = torch.randn((3, 4, 64), generator=torch.Generator(dev).manual_seed(1), device=dev)
    none = torch.zeros(3, dtype=torch.int32, device=dev)
    for n_pages, width in ((0, 0), (2, 0), (0, 3)):
        cache = nys.PagedKV4(n_pages, 16, 2, 64, 64, device=dev)
        table = torch.zeros((3, width), dtype=torch.int32, device=dev)
        out, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device=dev)
        att.paged4(q, cache, none, table, out, lse=lse)
        assert not bool(out.any()) and bool((lse == -math.inf).all()) and att.status() == 0
        first, first_lse = torch.randn_like(q), torch.randn_like(lse)
        att.paged4(q, cache, none, table, out, first=first, first_lse=first_lse, lse=lse)
        assert torch.allclose(out, first, rtol=1e-6) and torch.allclose(lse, first_lse, rtol=1e-5, atol=1e-6)
        # Lengths that nothing holds are taken as nothing, and said so.
        att.paged4(q, cache, none + 5, table, out)
        assert att.status() == (nys.NYS_ATTN_BAD_PAGE if width else nys.NYS_ATTN_BAD_LENGTH) and not bool(out.any())
        att.clear_status()
        cache.write(torch.zeros((2, 2, 64), device=dev), torch.zeros((2, 2, 64), device=dev),
                    torch.full((2,), -1, dtype=torch.int64, device=dev))
    empty = torch.empty((0, 4, 64), device=dev)
    assert att.paged4(empty, cache, none[:0], table[:0], empty) is empty
    rows = torch.empty((0, 2, 64), device=dev)
    cache.write(rows, rows, torch.empty(0, dtype=torch.int64, device=dev))
    cache.read(torch.empty(0, dtype=torch.int64, device=dev), rows, rows)
    prep = nys.QKPrepare(4, 2, 64, rotation=nys.Rotation(64, device=dev), device=dev)
    prep.rows(empty, rows, none[:0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[40000], [9000, 30011, 5], [1500] * 7])
def test_long_requests(cuda_device, dtype, lens):
    """Units cut into many pieces, of CTAs whose warps joined and of some that did not."""
    torch, ref, nys = _mods()
    dt, dev = getattr(torch, dtype), cuda_device
    for heads, kv, d in ((16, 2, 128), (4, 2, 64)):
        g = torch.Generator(device=dev).manual_seed(13)
        cache, table, slots = _cache(torch, nys, dev, g, lens, kv, d, d, 64, dt)
        q = torch.randn((len(lens), heads, d), generator=g, device=dev).to(dt)
        out, lse = torch.empty_like(q), torch.empty((len(lens), heads), device=dev)
        at = torch.tensor(lens, dtype=torch.int32, device=dev)
        att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=dev)
        att.paged4(q, cache, at, table, out, lse=lse)
        _check(torch, ref, cache, slots, q, out, lse, heads, 1 / math.sqrt(d), dt)


def test_many_keys_keep_their_digits(cuda_device):
    """Over 200,000 keys that have nothing in common the result is 1/270 of a value, and sums of
    one sign over that many would be 500 of it: what products cut off must not add up.  The
    result's own rounding is 2^-11 of each number at most, and a third of that squared on average: all
    errors together stay below 2^-11 if those of the sums are below 1.6 times the rounding's."""
    torch, ref, nys = _mods()
    dev, n, kv, d = cuda_device, 200000, 2, 128
    g = torch.Generator(device=dev).manual_seed(21)
    cache, table, slots = _cache(torch, nys, dev, g, [n], kv, d, d, 64, torch.float16)
    k, v = (torch.empty((n, kv, d), device=dev) for _ in range(2))
    nys.PagedKV4(*cache.data.shape[:1], 64, kv, d, d, device=dev, data=cache.data).read(slots[0].to(dev), k, v)
    at = torch.tensor([n], dtype=torch.int32, device=dev)
    for heads in (2, 4, 8, 16):
        q = torch.randn((1, heads, d), generator=g, device=dev).half()
        out = torch.empty_like(q)
        nys.ExactAttention(heads, kv, d, d, dtype=torch.float16, device=dev).paged4(q, cache, at, table, out)
        for h in range(heads):
            j = h // (heads // kv)
            p = (k[:, j].double() @ q[0, h].double() / math.sqrt(d)).softmax(0)
            want = p @ v[:, j].double()
            assert float((out[0, h].double() - want).norm() / want.norm()) <= 2.0 ** -11


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_large_queries(cuda_device, dtype):
    """Scores whose size no longer fits are NaN, never a result that looks like one; up to
    there the largest key wins."""
    torch, ref, nys = _mods()
    dt, dev = getattr(torch, dtype), cuda_device
    g = torch.Generator(device=dev).manual_seed(3)
    cache, table, _ = _cache(torch, nys, dev, g, [40], 1, 64, 64, 16, dt)
    at = torch.tensor([40], dtype=torch.int32, device=dev)
    k, v = (torch.empty((40, 1, 64), dtype=dt, device=dev) for _ in range(2))
    cache.read(table[0].repeat_interleave(16)[:40].long() * 16 + torch.arange(40, device=dev) % 16, k, v)
    att = nys.ExactAttention(1, 1, 64, 64, dtype=dt, device=dev, scale=1.0)
    for sign in (1.0, -1.0):
        for e in (60, 112, 118, 126):
            q = torch.zeros((1, 1, 64), dtype=dt, device=dev)
            q[..., 5] = sign * 2.0 ** e
            out = att.paged4(q, cache, at, table, torch.empty_like(q))
            right = torch.equal(out[0, 0], v[int((sign * k[:, 0, 5]).argmax()), 0])
            assert right or (e > 112 and bool(torch.isnan(out).all()))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("geo", [(14, 2, 80), (16, 8, 128), (32, 4, 128), (1, 1, 64)])
def test_single_keys_keep_their_digits(cuda_device, dtype, geo):
    """A request of one key: its log-sum is the score.  What is kept of a score is f32: a
    product a number, cut off by at most 2 U of the largest so far, of up to 128 (in f32
    calls queries to 2 U); on average over 200 scores far below 8 U of their terms' norm."""
    torch, ref, nys = _mods()
    heads, kv, d = geo
    dt, dev = getattr(torch, dtype), cuda_device
    g = torch.Generator(device=dev).manual_seed(17)
    n = 200 // heads + 1
    cache, table, slots = _cache(torch, nys, dev, g, [1] * n, kv, d, d, 16, dt)
    at = torch.ones(n, dtype=torch.int32, device=dev)
    q = torch.randn((n, heads, d), generator=g, device=dev).to(dt)
    lse = torch.empty((n, heads), device=dev)
    nys.ExactAttention(heads, kv, d, d, dtype=dt, device=dev).paged4(q, cache, at, table, torch.empty_like(q), lse=lse)
    (kc, ks, km), _ = ref.unpack(cache.data, kv, d, d, 16)
    k = ref.values(kc, ks, km)[torch.cat(slots)].repeat_interleave(heads // kv, 1)
    terms = q.double().cpu() * k / math.sqrt(d)
    off = (lse.double().cpu() - terms.sum(-1)).square().sum().sqrt()
    assert float(off) <= 8 * ref.U * float(terms.norm())


def test_wide_pool_offsets(cuda_device):
    """Pages whose bytes lie past 32 bits."""
    torch, ref, nys = _mods()
    kv, d, page = 8, 128, 128
    dev = cuda_device
    per = nys.nys_kv4_page_bytes(nys.NysAttnConfig(kv, kv, d, d, nys.NYS_BF16, 0.0), page)
    n_pages = (1 << 32) // per + 9
    cache = nys.PagedKV4(n_pages, page, kv, d, d, dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev).manual_seed(9)
    k, v = (torch.randn((130, kv, d), generator=g, device=dev).bfloat16() for _ in range(2))
    j = torch.arange(130, device=dev)
    pages = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device=dev)
    slots = pages[0].long()[j // page] * page + j % page
    cache.write(k, v, slots)
    small = nys.PagedKV4(2, page, kv, d, d, dtype=torch.bfloat16, device=dev)
    small.write(k, v, j)
    q = torch.randn((1, 16, d), generator=g, device=dev).bfloat16()
    att = nys.ExactAttention(16, kv, d, d, dtype=torch.bfloat16, device=dev)
    at = torch.tensor([130], dtype=torch.int32, device=dev)
    a = att.paged4(q, cache, at, pages, torch.empty_like(q))
    b = att.paged4(q, small, at, torch.tensor([[0, 1]], dtype=torch.int32, device=dev), torch.empty_like(q))
    assert torch.equal(a, b)
    x, y, z, w = (torch.empty_like(k) for _ in range(4))
    cache.read(slots, x, y)
    small.read(j, z, w)
    assert torch.equal(x, z) and torch.equal(y, w)


def test_capture_replay_and_two_graphs(cuda_device):
    """Graphs of two sizes over one object's workspace, replayed in turn with calls."""
    torch, ref, nys = _mods()
    heads, kv, d, page = 16, 8, 128, 16
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(10)
    att = nys.ExactAttention(heads, kv, d, d, dtype=torch.bfloat16, device=dev)
    sets = []
    for lens in ([700, 3], [90, 2000, 1, 64, 300]):
        cache, table, slots = _cache(torch, nys, dev, g, lens, kv, d, d, page, torch.bfloat16)
        q = torch.randn((len(lens), heads, d), generator=g, device=dev).bfloat16()
        at = torch.tensor(lens, dtype=torch.int32, device=dev)
        sets.append((q, cache, at, table, torch.empty_like(q)))
    graphs = []
    for q, cache, at, table, out in sets:
        att.paged4(q, cache, at, table, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            att.paged4(q, cache, at, table, out)
        graphs.append(graph)
    for _ in range(2):
        for graph, (q, cache, at, table, out) in zip(graphs, sets):
            q.copy_(torch.randn(q.shape, generator=g, device=dev))
            at.sub_(1)
            out.fill_(7.0)
            graph.replay()
            got = out.clone()
            att.paged4(q, cache, at, table, out)
            assert torch.equal(got, out)
    # The request of one token is at a length of -1 by now, and taken as empty.
    assert att.status() == nys.NYS_ATTN_BAD_LENGTH and not bool(sets[1][4][2].any())


def test_two_streams(cuda_device):
    """Two objects at work at once, each on a stream of its own."""
    torch, ref, nys = _mods()
    heads, kv, d, page = 8, 2, 128, 16
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(11)
    lens = [3000, 500, 7]
    cache, table, slots = _cache(torch, nys, dev, g, lens, kv, d, d, page, torch.float32)
    at = torch.tensor(lens, dtype=torch.int32, device=dev)
    q = torch.randn((2, 3, heads, d), generator=g, device=dev)
    atts = [nys.ExactAttention(heads, kv, d, d, device=dev) for _ in range(2)]
    want = [att.paged4(x, cache, at, table, torch.empty_like(x)) for att, x in zip(atts, q)]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(x) for _ in range(20)] for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(20):
        for s, att, x, o in zip(streams, atts, q, outs):
            with torch.cuda.stream(s):
                att.paged4(x, cache, at, table, o[i])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_refusals(cuda_device):
    torch, ref, nys = _mods()
    dev = cuda_device
    for bad in (dict(page=8), dict(page=24), dict(page=0)):
        with pytest.raises(ValueError):
            nys.PagedKV4(2, bad["page"], 2, 64, 64, device=dev)
    with pytest.raises(ValueError):
        nys.PagedKV4(2, 16, 2, 64, 64, device=dev, data=torch.zeros(10, dtype=torch.uint8, device=dev))
    cache = nys.PagedKV4(2, 16, 2, 64, 64, device=dev)
    z = lambda n, h, c=64: torch.zeros((n, h, c), device=dev)
    s = torch.zeros(3, dtype=torch.int64, device=dev)
    for call in (lambda: cache.write(z(3, 2), z(2, 2), s), lambda: cache.write(z(3, 2), z(3, 2), s.int()),
                 lambda: cache.write(z(3, 2).half(), z(3, 2), s), lambda: cache.read(s, z(2, 2), z(3, 2)),
                 lambda: cache.read(s, z(3, 2), z(3, 1))):
        with pytest.raises(ValueError):
            call()
    att = nys.ExactAttention(4, 2, 64, 64, device=dev)
    q, at, t = z(1, 4), torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros((1, 2), dtype=torch.int32, device=dev)
    lse = torch.zeros((1, 4), device=dev)
    full = nys.PagedKV(2, 16, 2, 64, 64, device=dev)
    for call in (lambda: att.paged4(q, full, at, t, z(1, 4)), lambda: att.paged4(q, cache, at, t, z(2, 4)),
                 lambda: att.paged4(q, cache, at, t[0], z(1, 4)), lambda: att.paged4(q, cache, at.long(), t, z(1, 4)),
                 lambda: att.paged4(q, cache, at, t, z(1, 4), first=q),
                 lambda: att.paged4(q, cache, at, t, z(1, 4), first_lse=lse),
                 lambda: att.paged4(q, nys.PagedKV4(2, 16, 1, 64, 64, device=dev), at, t, z(1, 4)),
                 lambda: att.shared(q, cache, at, t, z(1, 4))):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            call()
