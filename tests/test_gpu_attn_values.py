"""Exact attention on unusual values: what a row does not see never reaches it,
whatever it is, and what it sees reaches it as the formula says, against plain
64-bit forms (tests/attn_reference.py, where the bounds are derived)."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _mods():
    import torch
    import attn_reference as ref
    from streaming_nystr_landmark_gb300 import nys
    return torch, ref, nys


def _rand(torch, dev, rows, heads, kv, d, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda h: torch.randn((rows, h, d), generator=g, device=dev)
    return rn(heads), rn(kv), rn(kv)


def _prompt(torch, nys, q, k, v, q_lens, k_lens, scale=None):
    dev = q.device
    off = lambda x: torch.tensor([0] + x, device=dev).cumsum(0).int()
    att = nys.ExactAttention(q.shape[1], k.shape[1], q.shape[2], v.shape[2], dtype=q.dtype,
                             scale=scale, device=dev)
    out = torch.full((q.shape[0], q.shape[1], v.shape[2]), 7.0, device=dev, dtype=q.dtype)
    lse = torch.full(out.shape[:2], 7.0, device=dev)
    att.prompt(q, k, v, off(q_lens), out, k_off=off(k_lens), lse=lse)
    assert att.status() == 0
    return out, lse


def test_long_row_of_nan_beside_healthy_ones(cuda_device):
    """400,000 values that are not finite in a unit that is not cut (129 sequences
    and more): it is slow, and nothing gives up waiting for it."""
    torch, ref, nys = _mods()
    n, long, d = 130, 400000, 64
    q_lens, k_lens = [1] + [3] * (n - 1), [long] + [3] * (n - 1)
    q, _, _ = _rand(torch, cuda_device, sum(q_lens), 1, 1, d)
    _, k, v = _rand(torch, cuda_device, sum(k_lens), 1, 1, d, seed=1)
    v[:long] = math.nan
    out, lse = _prompt(torch, nys, q, k, v, q_lens, k_lens)
    assert bool(torch.isnan(out[0]).all())
    want = torch.logsumexp(k[:long, 0].double() @ q[0, 0].double() / 8.0, 0)
    assert abs(float(lse[0, 0]) - float(want)) < 1e-4
    want, wl, b, lb = ref.prompt(q[1:], k[long:], v[long:], [3] * (n - 1), [3] * (n - 1), 1, 1 / 8.0,
                                 torch.float32)
    ref.check(out[1:], want, b, "out")
    ref.check(lse[1:], wl, lb, "lse")


@pytest.mark.parametrize("geo", [(4, 2, 128), (3, 1, 20), (40, 1, 64)])
@pytest.mark.parametrize("q_len,k_len", [(150, 150), (40, 333), (1, 2000), (200, 90)])
def test_f32_units_with_bad_values(cuda_device, geo, q_len, k_len):
    """One infinity far from most rows: its own channel of the rows that see it,
    and everything else, log-sums among it, as without it."""
    torch, ref, nys = _mods()
    heads, kv, d = geo
    q, _, _ = _rand(torch, cuda_device, q_len, heads, kv, d)
    _, k, v = _rand(torch, cuda_device, k_len, heads, kv, d, seed=1)
    want, wl, b, lb = ref.prompt(q, k, v, [q_len], [k_len], heads // kv, 1 / math.sqrt(d),
                                 torch.float32)
    at = k_len - 17
    v[at, kv - 1, 5] = math.inf
    out, lse = _prompt(torch, nys, q, k, v, [q_len], [k_len])
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[max(0, at + q_len - k_len):, heads - heads // kv:, 5] = True
    got = out.cpu()
    assert not bool(torch.isfinite(got[hit]).any())
    ref.check(got[~hit], want[~hit], b[~hit], "out")
    ref.check(lse, wl, lb, "lse")


def _without(torch, ref, q, k, v, q_lens, gone, group):
    """The plain form of one sequence in which no row gives key `gone` any weight."""
    n = k.shape[0]
    d = q.shape[2]
    i, j = torch.arange(q_lens)[:, None], torch.arange(n)[None, :]
    seen = (j <= i + n - q_lens) & (j != gone)
    res = [ref.attend(q[:, h].double().cpu(), k[:, h // group].double().cpu(),
                      v[:, h // group].double().cpu(), seen, 1 / math.sqrt(d), q.dtype)
           for h in range(q.shape[1])]
    return [torch.stack([r[x] for r in res], 1) for x in range(4)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("q_len,k_len", [(64, 64), (1, 300), (150, 400), (1, 3000)])
def test_key_of_minus_infinity_has_no_weight(cuda_device, dtype, q_len, k_len):
    """An infinite element against queries that give the score -inf."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, at = 4, 2, 64, 10
    q, _, _ = _rand(torch, cuda_device, q_len, heads, kv, d)
    _, k, v = _rand(torch, cuda_device, k_len, heads, kv, d, seed=1)
    q[..., 5] = q[..., 5].abs() + 0.1
    q[..., 9] = -q[..., 9].abs() - 0.1
    q, k, v = q.to(dt), k.to(dt), v.to(dt)
    want, wl, b, lb = _without(torch, ref, q, k, v, q_len, at, heads // kv)
    k[at, 0, 5], k[at, 1, 9] = -math.inf, math.inf
    out, lse = _prompt(torch, nys, q, k, v, [q_len], [k_len])
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")


def test_prefix_key_of_minus_infinity_has_no_weight(cuda_device):
    """The same for keys of a prefix that is read once for all requests (f32)."""
    torch, ref, nys = _mods()
    n, heads, kv, d, page, prefix = 300, 4, 2, 64, 16, 512
    q, _, _ = _rand(torch, cuda_device, n, heads, kv, d)
    _, k, v = _rand(torch, cuda_device, prefix, heads, kv, d, seed=1)
    q[..., 5] = q[..., 5].abs() + 0.1
    rest = [x for x in range(prefix) if x != 200]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    want = [ref.attend(q[:, h].double().cpu(), k[rest, h // 2].double().cpu(),
                       v[rest, h // 2].double().cpu(), torch.ones(n, prefix - 1, dtype=torch.bool),
                       1 / 8.0, torch.float32) for h in range(heads)]
    k[200, :, 5] = -math.inf
    cache = nys.PagedKV(prefix // page, page, kv, d, d, device=cuda_device,
                        k=k.view(-1, page, kv, d), v=v.view(-1, page, kv, d))
    att = nys.ExactAttention(heads, kv, d, d, device=cuda_device)
    out = torch.empty((n, heads, d), device=cuda_device)
    att.shared(q, cache, i32([0] * n), i32([[0]] * n), out,
               prefix_pages=i32(list(range(prefix // page))), prefix_len=prefix)
    ref.check(out, torch.stack([w[0] for w in want], 1), torch.stack([w[2] for w in want], 1), "out")
    assert att.status() == 0


@pytest.mark.parametrize("size", [1e10, 1.0, 1e-2, 1e-4, 1e-6, 1e-8, 1e-12, 1e-20])
@pytest.mark.parametrize("q_len,k_len", [(64, 64), (1, 200), (100, 700)])
def test_zero_values_beside_small_ones(cuda_device, size, q_len, k_len):
    """16 zero value rows: they take their share of the weight and nothing else."""
    torch, ref, nys = _mods()
    heads, kv, d = 2, 1, 64
    q, _, _ = _rand(torch, cuda_device, q_len, heads, kv, d)
    _, k, v = _rand(torch, cuda_device, k_len, heads, kv, d, seed=1)
    v *= size
    v[16:32] = 0
    want, wl, b, lb = ref.prompt(q, k, v, [q_len], [k_len], heads, 1 / math.sqrt(d), torch.float32)
    out, lse = _prompt(torch, nys, q, k, v, [q_len], [k_len])
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")


@pytest.mark.parametrize("size", [1.0, 1e-6, 1e-20])
def test_zero_pages_of_a_prefix_of_small_values(cuda_device, size):
    """The same for a prefix read once for all requests (f32); a page outside the
    pool counts as zeros."""
    torch, ref, nys = _mods()
    n, heads, kv, d, page, prefix = 300, 4, 2, 64, 16, 512
    q, _, _ = _rand(torch, cuda_device, n, heads, kv, d)
    _, k, v = _rand(torch, cuda_device, prefix, heads, kv, d, seed=1)
    v *= size
    v[64:80] = 0
    pages = list(range(prefix // page))
    pages[7] = 1 << 20
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    pk, pv = k.view(-1, page, kv, d), v.view(-1, page, kv, d)
    want, wl, b, lb = ref.shared(q, pk, pv, pages, prefix, [0] * n, [[0]] * n, heads // kv, 1 / 8.0,
                                 torch.float32)
    cache = nys.PagedKV(prefix // page, page, kv, d, d, device=cuda_device, k=pk, v=pv)
    att = nys.ExactAttention(heads, kv, d, d, device=cuda_device)
    out, lse = torch.empty((n, heads, d), device=cuda_device), torch.empty((n, heads), device=cuda_device)
    att.shared(q, cache, i32([0] * n), i32([[0]] * n), out, prefix_pages=i32(pages),
               prefix_len=prefix, lse=lse)
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")
    assert att.status() == nys.NYS_ATTN_BAD_PAGE


SIZES = [2.0 ** e for e in (4, 8, 10, 12, 13, 14, 16, 20, 40)] + [1e6, 1e12, 1e30]


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("n,at", [(48, 10), (300, 290), (500, 127)])
def test_f32_large_values_that_rows_do_not_see(cuda_device, what, size, n, at):
    """A key's finite row, far larger than those before it: rows that do not see
    it come out as if it were ordinary, in its group of keys, its tile and beyond."""
    torch, ref, nys = _mods()
    heads, kv, d = 2, 1, 64
    q, k, v = _rand(torch, cuda_device, n, heads, kv, d)
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads, 1 / math.sqrt(d), torch.float32)
    (k if what == "k" else v)[at] *= size
    out, lse = _prompt(torch, nys, q, k, v, [n], [n])
    ref.check(out[:at], want[:at], b[:at], "out")
    ref.check(lse[:at], wl[:at], lb[:at], "lse")
    if what == "v":   # and the others as the formula says
        want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads, 1 / math.sqrt(d), torch.float32)
        ref.check(out, want, b, "out")
        ref.check(lse, wl, lb, "lse")


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("rows", [slice(10, 11), slice(32, 48), slice(128, 300), slice(3, 300, 2)])
def test_f32_large_values_that_rows_see(cuda_device, size, rows):
    """Large value rows among ordinary ones, with weights of their own: one, a
    group of keys, whole tiles, every other one."""
    torch, ref, nys = _mods()
    n, heads, kv, d = 300, 2, 1, 64
    q, k, v = _rand(torch, cuda_device, n, heads, kv, d)
    v[rows] *= size
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads, 1 / math.sqrt(d), torch.float32)
    out, lse = _prompt(torch, nys, q, k, v, [n], [n])
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("score", [-4.0, -12.0, -30.0, -60.0])
def test_f32_large_value_of_small_weight(cuda_device, size, score):
    """One large value row whose key's score is far below the others'."""
    torch, ref, nys = _mods()
    n, heads, kv, d = 200, 1, 1, 64
    q, _, _ = _rand(torch, cuda_device, 1, heads, kv, d)
    _, k, v = _rand(torch, cuda_device, n, heads, kv, d, seed=1)
    k[77, 0] = q[0, 0] * (score * math.sqrt(d)) / float(q[0, 0] @ q[0, 0])
    v[77] *= size
    want, wl, b, lb = ref.prompt(q, k, v, [1], [n], 1, 1 / math.sqrt(d), torch.float32)
    out, lse = _prompt(torch, nys, q, k, v, [1], [n])
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")


@pytest.mark.parametrize("size", SIZES + [1 / x for x in SIZES])
@pytest.mark.parametrize("where", ["v one", "v column", "k column", "k one", "q column", "q one"])
def test_f32_columns_of_other_sizes(cuda_device, size, where):
    """One element, or one column, far from the rest; where it is the keys' or the
    queries' the other side's column makes up for it, so that scores stay ordinary."""
    torch, ref, nys = _mods()
    n, heads, kv, d, c = 200, 2, 1, 64, 13
    q, k, v = _rand(torch, cuda_device, n, heads, kv, d)
    if where == "v one":
        v[20, 0, c] *= size
    elif where == "v column":
        v[..., c] *= size
    elif where in ("k column", "q column"):
        x = size if where[0] == "k" else 1 / size
        k[..., c] *= x
        q[..., c] /= x
    elif where == "k one":
        k[20, 0, c] *= size
        q[..., c] *= 1 / size if size > 1 else 1.0
    else:
        q[20, :, c] *= size
        k[..., c] *= 1 / size if size > 1 else 1.0
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads, 1 / math.sqrt(d), torch.float32)
    out, lse = _prompt(torch, nys, q, k, v, [n], [n])
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")


@pytest.mark.parametrize("size", [1e6, 1e12, 1e30])
@pytest.mark.parametrize("where", ["row", "column", "own pages"])
def test_f32_shared_prefix_of_other_sizes(cuda_device, size, where):
    """A prefix read once for all requests, and own pages beside it."""
    torch, ref, nys = _mods()
    n, heads, kv, d, page, prefix = 300, 4, 2, 64, 16, 512
    q, _, _ = _rand(torch, cuda_device, n, heads, kv, d)
    _, k, v = _rand(torch, cuda_device, prefix + n * page, heads, kv, d, seed=1)
    if where == "row":
        v[100] *= size
    elif where == "column":
        v[:prefix, :, 3] *= size
    else:
        v[prefix::2] *= size
    pk, pv = k.view(-1, page, kv, d), v.view(-1, page, kv, d)
    pages = list(range(prefix // page))
    table, lens = [[prefix // page + i] for i in range(n)], [i % 17 for i in range(n)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    want, wl, b, lb = ref.shared(q, pk, pv, pages, prefix, lens, table, heads // kv, 1 / 8.0,
                                 torch.float32)
    cache = nys.PagedKV(pk.shape[0], page, kv, d, d, device=cuda_device, k=pk, v=pv)
    att = nys.ExactAttention(heads, kv, d, d, device=cuda_device)
    out, lse = torch.empty((n, heads, d), device=cuda_device), torch.empty((n, heads), device=cuda_device)
    att.shared(q, cache, i32(lens), i32(table), out, prefix_pages=i32(pages), prefix_len=prefix,
               lse=lse)
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")
    assert att.status() == 0


def test_f32_call_without_units_before_another(cuda_device):
    """Rows that no sequence covers: the attention launch has nothing to do but is
    not done before its keys' split is, whose workspace the next call takes."""
    torch, ref, nys = _mods()
    heads, kv, d, n = 4, 2, 64, 3000
    q, k, v = _rand(torch, cuda_device, n, heads, kv, d)
    q2, k2, v2 = _rand(torch, cuda_device, 200, heads, kv, d, seed=1)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    want, _, b, _ = ref.prompt(q2, k2, v2, [200], [200], 2, 1 / 8.0, torch.float32)
    att = nys.ExactAttention(heads, kv, d, d, device=cuda_device)
    none, koff, off, out = i32(0, 0), i32(0, n), i32(0, 200), torch.full_like(q, 7.0)
    got = [torch.empty_like(q2) for _ in range(20)]
    for x in got:
        att.prompt(q, k, v, none, out, k_off=koff)
        att.prompt(q2, k2, v2, off, x)
    assert bool((out == 7.0).all())
    for x in got:
        assert torch.equal(x, got[0])
    ref.check(got[0], want, b, "out")
    assert att.status() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("gap", [10.0, 14.0, 17.4, 20.0])
@pytest.mark.parametrize("how", ["prompt", "prompt cut", "pages", "prefix"])
def test_many_keys_of_small_weight(cuda_device, dtype, gap, how):
    """One key far above all others, with value 0: the result is the others' share.
    A weight is off by half a step, or by half of fp16's smallest step at 2^7
    (2^-32 of the largest); sums and the exponential as in attn_reference."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    n, d, page = 4096 if how == "prompt cut" else 1472, 64, 16
    q = torch.zeros(1, 1, d, device=cuda_device, dtype=dt)
    k = torch.zeros(n, 1, d, device=cuda_device, dtype=dt)
    v = torch.ones(n, 1, d, device=cuda_device, dtype=dt)
    q[..., 0], k[0, 0, 0], v[0] = 1, gap, 0
    att = nys.ExactAttention(1, 1, d, d, dtype=dt, scale=1.0, device=cuda_device)
    requests = 300 if how == "prefix" else 1
    out = torch.empty(requests, 1, d, device=cuda_device, dtype=dt)
    lse = torch.empty(requests, 1, device=cuda_device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    if how.startswith("prompt"):
        att.prompt(q, k, v, i32([0, 1]), out, k_off=i32([0, n]), lse=lse)
    else:
        cache = nys.PagedKV(n // page, page, 1, d, d, dtype=dt, device=cuda_device,
                            k=k.view(-1, page, 1, d), v=v.view(-1, page, 1, d))
        pages = list(range(n // page))
        if how == "pages":
            att.shared(q, cache, i32([n]), i32([pages]), out, lse=lse)
        else:
            att.shared(q.expand(requests, 1, d).contiguous(), cache, i32([0] * requests),
                       i32([[0]] * requests), out, prefix_pages=i32(pages), prefix_len=n, lse=lse)
    w = math.exp(-float(k[0, 0, 0]))
    total = 1 + (n - 1) * w
    want = (n - 1) * w / total
    half = 0.0 if dtype == "float32" else ref.EPS[dt]
    weight = max(w * half, 2.0 ** -32 if dtype == "float16" else 0.0)
    bound = ((n - 1) * weight / total + want * (ref.EPS[dt] + 2.0 ** -18 + n * 2.0 ** -23)
             + (2.0 ** -25 if dtype == "float16" else 0.0))
    err = float((out.double() - want).abs().max())
    assert err <= bound, (err, bound, want)
    assert float((lse.double() - float(k[0, 0, 0]) - math.log(total)).abs().max()) < 2.0 ** -17
    assert att.status() == 0


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("rows", [slice(16, 32), slice(128, 256)])
def test_f32_large_values_without_a_column(cuda_device, size, rows):
    """A group of keys, or a tile, of large values that has nothing in one column:
    there the other keys' values are all there is."""
    torch, ref, nys = _mods()
    n, heads, kv, d = 300, 2, 1, 64
    q, k, v = _rand(torch, cuda_device, n, heads, kv, d)
    v[rows] *= size
    v[rows, :, 3] = 0
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads, 1 / math.sqrt(d), torch.float32)
    out, lse = _prompt(torch, nys, q, k, v, [n], [n])
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")


@pytest.mark.parametrize("d", [4, 8, 20])
@pytest.mark.parametrize("n", [1, 2, 7, 30])
@pytest.mark.parametrize("size", [1e6, 1e12, 1e18])
@pytest.mark.parametrize("where", ["one column", "every fourth", "a diagonal"])
def test_f32_few_numbers_of_other_sizes(cuda_device, d, n, size, where):
    """Narrow and short: every row, every column and every four numbers may hold a
    large one."""
    torch, ref, nys = _mods()
    q, k, v = _rand(torch, cuda_device, n, 2, 1, d)
    if where == "one column":
        v[..., 1] *= size
    elif where == "every fourth":
        v[..., ::4] *= size
    else:
        for i in range(n):
            v[i, :, i % 4::4] *= size
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], 2, 1 / math.sqrt(d), torch.float32)
    out, lse = _prompt(torch, nys, q, k, v, [n], [n])
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")
