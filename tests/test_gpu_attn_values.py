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
