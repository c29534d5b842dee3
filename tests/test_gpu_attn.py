"""Exact attention, block tables and page writes on the GPU against plain
64-bit forms (tests/attn_reference.py, where the bounds are derived)."""
import math

import pytest

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]
GEOMETRIES = [(1, 1, 64, 64), (16, 8, 128, 128), (8, 1, 128, 128), (6, 2, 96, 64),
              (14, 2, 80, 128), (2, 2, 20, 12), (4, 2, 192, 256)]


def _mods():
    import torch
    import attn_reference as ref
    from streaming_nystr_landmark_gb300 import nys
    return torch, ref, nys


def _inputs(torch, dev, q_lens, k_lens, heads, kv, d, dv, dtype, seed=0, big=1.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=dev)
    u = rn(1, kv, d)
    q = (rn(sum(q_lens), heads, d) * big).to(dtype)
    k = (rn(sum(k_lens), kv, d) + 2 * u / u.norm(dim=-1, keepdim=True)).to(dtype)
    v = rn(sum(k_lens), kv, dv).to(dtype)
    off = lambda x: torch.tensor([0] + x, device=dev).cumsum(0).int()
    return q, k, v, off(q_lens), off(k_lens)


def _run_prompt(cuda_device, dtype, geo, q_lens, k_lens, scale=None, big=1.0, seed=0, edit=None):
    torch, ref, nys = _mods()
    heads, kv, d, dv = geo
    dtype = getattr(torch, dtype)
    q, k, v, qo, ko = _inputs(torch, cuda_device, q_lens, k_lens, heads, kv, d, dv, dtype, seed, big)
    if edit:
        edit(q, k, v)
    att = nys.ExactAttention(heads, kv, d, dv, dtype=dtype, scale=scale, device=cuda_device)
    out = torch.full((q.shape[0], heads, dv), 7.0, device=cuda_device, dtype=dtype)
    lse = torch.full(out.shape[:2], 7.0, device=cuda_device)
    att.prompt(q, k, v, qo, out, k_off=ko, lse=lse)
    want, wl, b, lb = ref.prompt(q, k, v, q_lens, k_lens, heads // kv,
                                 1 / math.sqrt(d) if scale is None else scale, dtype)
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")
    assert att.status() == 0
    return q, k, v, out, lse


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("geo", GEOMETRIES)
def test_prompt_geometries(cuda_device, dtype, geo):
    lens = [1, 0, 130, 7, 64]
    _run_prompt(cuda_device, dtype, geo, lens, lens)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_lens,k_lens", [
    ([1], [1]), ([127], [127]), ([128], [128]), ([129], [129]), ([255, 257], [255, 257]),
    ([640], [640]), ([1, 1, 1], [1, 500, 129]), ([3, 200], [900, 333]),
    ([0, 5], [17, 0]), ([300], [40]), ([140, 9], [128, 256]), ([1], [3000])])
def test_prompt_lengths(cuda_device, dtype, q_lens, k_lens):
    """Continued prompts, single tokens, and queries that see no key."""
    _run_prompt(cuda_device, dtype, (16, 8, 128, 128), q_lens, k_lens)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_many_sequences(cuda_device, dtype):
    lens = [(i * 37) % 53 for i in range(700)]
    _run_prompt(cuda_device, dtype, (4, 2, 64, 64), lens, lens)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_large_scores_and_scale(cuda_device, dtype):
    """Scores in the hundreds: one key holds nearly all the weight."""
    _run_prompt(cuda_device, dtype, (8, 2, 128, 128), [300], [300], scale=1.0, big=6.0)
    _run_prompt(cuda_device, dtype, (8, 2, 128, 128), [300], [300], scale=1e-3)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_values_of_other_magnitudes(cuda_device, dtype):
    """Rows of very large and very small keys and values side by side."""
    def edit(q, k, v):
        v[40:60] *= 1e-4
        v[200:210] *= 3e3
        k[100:180] *= 1e-3
        q[30:50] *= 1e-2
    _run_prompt(cuda_device, dtype, (4, 2, 128, 128), [333], [333], edit=edit)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [40, 200, 400])
def test_prompt_unseen_rows_do_not_matter(cuda_device, dtype, bad, n):
    """NaN and infinities in later keys and values, and in other sequences'
    rows, reach no row that does not see them."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d = 8, 2, 128
    lens = [n, 33]
    q, k, v, qo, ko = _inputs(torch, cuda_device, lens, lens, heads, kv, d, d, dt)
    want, wl, b, lb = ref.prompt(q, k, v, lens, lens, heads // kv, 1 / math.sqrt(d), dt)
    cut = n - 13
    k[cut:n], v[cut:n] = bad, bad
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda_device)
    att.prompt(q, k, v, qo, out, lse=lse)
    keep = list(range(cut)) + list(range(n, n + 33))
    ref.check(out[keep], want[keep], b[keep], "out")
    ref.check(lse[keep], wl[keep], lb[keep], "lse")
    # Rows that see them say so.
    assert not torch.isfinite(out[cut + 1:n].float()).all(dim=-1).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prompt_seen_bad_values(cuda_device, dtype, bad):
    """A value that is not finite reaches exactly its own channel of the rows
    that see its key."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, n = 4, 2, 128, 300
    q, k, v, qo, ko = _inputs(torch, cuda_device, [n], [n], heads, kv, d, d, dt)
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads // kv, 1 / math.sqrt(d), dt)
    spots = [(5, 0, 3), (150, 1, 70), (290, 0, 127)]
    for j, g, c in spots:
        v[j, g, c] = bad
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out = torch.empty_like(q)
    att.prompt(q, k, v, qo, out)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    for j, g, c in spots:
        hit[j:, g * 2:g * 2 + 2, c] = True
    got = out.float().cpu()
    assert not torch.isfinite(got[hit]).any()
    ref.check(got[~hit], want[~hit], b[~hit], "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("how", ["heads first", "padded rows", "one base", "odd start"])
def test_prompt_strides(cuda_device, dtype, how):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, n = 6, 2, 64, 150
    q, k, v, qo, ko = _inputs(torch, cuda_device, [n], [n], heads, kv, d, d, dt)
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads // kv, 1 / math.sqrt(d), dt)
    out = torch.zeros_like(q)
    if how == "heads first":
        swap = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
        q, k, v, out = swap(q), swap(k), swap(v), swap(out)
    elif how == "padded rows":
        def pad(t, extra):
            big = torch.full((t.shape[0], t.shape[1], t.shape[2] + extra), math.nan,
                             device=t.device, dtype=dt)
            big[..., :t.shape[2]] = t
            return big[..., :t.shape[2]]
        q, k, v, out = pad(q, 8), pad(k, 3), pad(v, 16), pad(out, 5)
    elif how == "one base":
        qkv = torch.cat([q, k, v], dim=1)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    else:
        def shift(t):
            flat = torch.empty(t.numel() + 1, device=t.device, dtype=dt)
            flat[1:] = t.reshape(-1)
            return flat[1:].view(t.shape)
        q, k, v, out = shift(q), shift(k), shift(v), shift(out)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    att.prompt(q, k, v, qo, out)
    ref.check(out, want, b, how)


def test_prompt_shared_kv_heads_broadcast(cuda_device):
    """A KV tensor expanded over heads (head stride 0) is read in place."""
    torch, ref, nys = _mods()
    n, heads, d = 70, 4, 64
    q, k, v, qo, ko = _inputs(torch, cuda_device, [n], [n], heads, 1, d, d, torch.bfloat16)
    want, wl, b, lb = ref.prompt(q, k, v, [n], [n], heads, 1 / math.sqrt(d), torch.bfloat16)
    att = nys.ExactAttention(heads, 2, d, d, dtype=torch.bfloat16, device=cuda_device)
    out = torch.empty_like(q)
    att.prompt(q, k.expand(n, 2, d), v.expand(n, 2, d), qo, out)
    ref.check(out, want, b, "out")


def test_prompt_bad_offsets_are_clamped_and_reported(cuda_device):
    torch, ref, nys = _mods()
    n, heads, d = 64, 2, 64
    q, k, v, _, _ = _inputs(torch, cuda_device, [n], [n], heads, 2, d, d, torch.float32)
    att = nys.ExactAttention(heads, 2, d, d, device=cuda_device)
    out = torch.zeros_like(q)
    qo = torch.tensor([0, 20, 90], device=cuda_device, dtype=torch.int32)
    att.prompt(q, k, v, qo, out)
    assert att.status() == nys.NYS_ATTN_BAD_OFFSETS
    att.clear_status()
    want, _, b, _ = ref.prompt(q, k, v, [20, 44], [20, 44], 1, 1 / 8.0, torch.float32)
    ref.check(out, want, b, "out")
    att.prompt(q, k, v, torch.tensor([-5, 40, 30], device=cuda_device, dtype=torch.int32), out)
    assert att.status() == nys.NYS_ATTN_BAD_OFFSETS


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_on_another_stream_and_in_a_graph(cuda_device, dtype):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    lens = [200, 3]
    q, k, v, qo, ko = _inputs(torch, cuda_device, lens, lens, 4, 2, 128, 128, dt)
    want, wl, b, lb = ref.prompt(q, k, v, lens, lens, 2, 1 / math.sqrt(128), dt)
    att = nys.ExactAttention(4, 2, 128, 128, dtype=dt, device=cuda_device)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        att.prompt(q, k, v, qo, out)
    side.synchronize()
    ref.check(out, want, b, "other stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.prompt(q, k, v, qo, out)
    q2, k2, v2, _, _ = _inputs(torch, cuda_device, lens, lens, 4, 2, 128, 128, dt, seed=5)
    q.copy_(q2), k.copy_(k2), v.copy_(v2)
    out.zero_()
    graph.replay()
    want, wl, b, lb = ref.prompt(q, k, v, lens, lens, 2, 1 / math.sqrt(128), dt)
    ref.check(out, want, b, "replayed")


def test_prompt_same_bits_every_time(cuda_device):
    torch, ref, nys = _mods()
    lens = [513, 77, 1200]
    for dt in (torch.float32, torch.bfloat16):
        q, k, v, qo, ko = _inputs(torch, cuda_device, lens, lens, 8, 2, 128, 128, dt)
        att = nys.ExactAttention(8, 2, 128, 128, dtype=dt, device=cuda_device)
        a, b = torch.empty_like(q), torch.empty_like(q)
        att.prompt(q, k, v, qo, a)
        for _ in range(5):
            att.prompt(q, k, v, qo, b)
            assert torch.equal(a, b)


# ------------------------------------------------------------------ shared
def _pool(torch, dev, lens, prefix, page, kv, d, dv, dtype, seed=0, junk=math.nan):
    """A pool whose unused slots hold `junk`, with shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    first, need = -(-prefix // page), [-(-x // page) for x in lens]
    n_pages = first + sum(need) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    k = torch.full((n_pages, page, kv, d), junk)
    v = torch.full((n_pages, page, kv, dv), junk)
    u = torch.randn((kv, d), generator=g)

    def fill(pages, count):
        for x in range(count):
            p, o = pages[x // page], x % page
            k[p, o] = torch.randn((kv, d), generator=g) + 2 * u / u.norm(dim=-1, keepdim=True)
            v[p, o] = torch.randn((kv, dv), generator=g)

    pp, at, width = order[:first], first, max(need + [1])
    fill(pp, prefix)
    table = [[-1] * width for _ in lens]
    for i, x in enumerate(need):
        table[i][:x] = order[at:at + x]
        fill(table[i], lens[i])
        at += x
    return k.to(dtype).to(dev), v.to(dtype).to(dev), pp, table


def _run_shared(cuda_device, dtype, geo, lens, prefix, page, seed=0):
    torch, ref, nys = _mods()
    heads, kv, d, dv = geo
    dt = getattr(torch, dtype)
    k, v, pp, table = _pool(torch, cuda_device, lens, prefix, page, kv, d, dv, dt, seed)
    q = torch.randn((len(lens), heads, d), device=cuda_device).to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cache = nys.PagedKV(k.shape[0], page, kv, d, dv, dtype=dt, device=cuda_device, k=k, v=v)
    att = nys.ExactAttention(heads, kv, d, dv, dtype=dt, device=cuda_device)
    out = torch.full((len(lens), heads, dv), 7.0, device=cuda_device, dtype=dt)
    lse = torch.full((len(lens), heads), 7.0, device=cuda_device)
    att.shared(q, cache, i32(lens), i32(table), out, prefix_pages=i32(pp), prefix_len=prefix, lse=lse)
    want, wl, b, lb = ref.shared(q, k, v, pp, prefix, lens, table, heads // kv, 1 / math.sqrt(d), dt)
    ref.check(out, want, b, "out")
    ref.check(lse, wl, lb, "lse")
    assert att.status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("geo", GEOMETRIES)
def test_shared_geometries(cuda_device, dtype, geo):
    _run_shared(cuda_device, dtype, geo, [5, 40, 1], 50, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,prefix,page", [
    ([0], 0, 16), ([0, 3], 0, 16), ([0, 0], 9, 16), ([1], 1, 1), ([17, 16, 15, 32, 33], 129, 16),
    ([63, 64, 65], 128, 64), ([100, 7], 127, 24), ([130, 257, 3], 300, 8), ([9, 2], 1000, 7),
    ([700, 1], 5, 128), ([3] * 150, 260, 16), ([1500], 0, 32), ([40], 2100, 16)])
def test_shared_lengths(cuda_device, dtype, lens, prefix, page):
    """Pages that end inside a tile, empty requests, no prefix; what lies past
    a length in its page is NaN."""
    _run_shared(cuda_device, dtype, (16, 8, 128, 128), lens, prefix, page)


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_many_query_rows(cuda_device, dtype):
    """More rows a KV head than one tile holds."""
    _run_shared(cuda_device, dtype, (8, 1, 64, 64), [(i * 7) % 40 for i in range(70)], 333, 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_bad_pages_and_lengths(cuda_device, dtype):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, page = 4, 2, 64, 8
    lens, prefix = [20, 30], 40
    k, v, pp, table = _pool(torch, cuda_device, lens, prefix, page, kv, d, d, dt, junk=0.0)
    pp[1], table[0][0], table[1][2] = k.shape[0], -1, 1 << 30
    q = torch.randn((2, heads, d), device=cuda_device).to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cache = nys.PagedKV(k.shape[0], page, kv, d, d, dtype=dt, device=cuda_device, k=k, v=v)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out = torch.empty((2, heads, d), device=cuda_device, dtype=dt)
    att.shared(q, cache, i32(lens), i32(table), out, prefix_pages=i32(pp), prefix_len=prefix)
    want, _, b, _ = ref.shared(q, k, v, pp, prefix, lens, table, 2, 1 / 8.0, dt)
    ref.check(out, want, b, "out")
    assert att.status() == nys.NYS_ATTN_BAD_PAGE
    att.clear_status()
    # Lengths outside the table are clamped to it.
    table[0][0], table[1][2], pp[1] = 0, 1, 2
    att.shared(q, cache, i32([-3, 1000]), i32(table), out, prefix_pages=i32(pp), prefix_len=prefix)
    want, _, b, _ = ref.shared(q, k, v, pp, prefix, [0, len(table[1]) * page], table, 2, 1 / 8.0, dt)
    ref.check(out, want, b, "out")
    assert att.status() & nys.NYS_ATTN_BAD_LENGTH
    att.clear_status()


def test_shared_offsets_past_32_bits(cuda_device):
    """A pool of more than 2^32 elements: pages at its far end."""
    torch, ref, nys = _mods()
    page, kv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * kv * d) + 40
    k = torch.empty((n_pages, page, kv, d), dtype=torch.bfloat16, device=cuda_device)
    v = torch.empty_like(k)
    pages = [n_pages - 1, n_pages - 7, n_pages - 3]
    for p in pages:
        k[p].normal_(), v[p].normal_()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cache = nys.PagedKV(n_pages, page, kv, d, d, dtype=torch.bfloat16, device=cuda_device, k=k, v=v)
    new = torch.randn((1, kv, d), device=cuda_device).bfloat16()
    cache.write(new, new, torch.tensor([pages[1] * page + 36], device=cuda_device))
    assert torch.equal(k[pages[1], 36], new[0])
    q = torch.randn((2, 16, d), device=cuda_device).bfloat16()
    att = nys.ExactAttention(16, kv, d, d, dtype=torch.bfloat16, device=cuda_device)
    out = torch.empty_like(q)
    att.shared(q, cache, i32([37, 64]), i32([[pages[1]], [pages[2]]]), out,
               prefix_pages=i32([pages[0]]), prefix_len=60)
    few = torch.tensor(pages, device=cuda_device)
    want, _, b, _ = ref.shared(q, k[few], v[few], [0], 60, [37, 64], [[1], [2]], 2,
                               1 / math.sqrt(d), torch.bfloat16)
    ref.check(out, want, b, "out")


# ------------------------------------------------------------ plan and write
@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("n,most_cached,most_fresh", [(1, 0, 1), (5, 40, 0), (64, 300, 1),
                                                      (33, 0, 90), (3000, 20, 5), (2, 9000, 4100)])
def test_plan(cuda_device, page, n, most_cached, most_fresh):
    torch, ref, nys = _mods()
    g = torch.Generator().manual_seed(n + page)
    rnd = lambda most: torch.randint(0, most + 1, (n,), generator=g).tolist()
    cached, fresh = rnd(most_cached), rnd(most_fresh)
    old = [-(-c // page) for c in cached]
    new = [-(-(c + f) // page) for c, f in zip(cached, fresh)]
    order = torch.randperm(sum(new) + 3, generator=g).tolist()
    width = max(new + [1])
    table, at = [], 0
    for o in old:
        table.append(order[at:at + o] + [-1] * (width - o))
        at += o
    free = order[at:]
    want = ref.plan(cached, fresh, free, table, page)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    t = i32(table)
    p = nys.PagePlan(n, width, sum(fresh), page, device=cuda_device)
    for _ in range(2):   # a second run changes nothing
        p.update(i32(cached), i32(fresh), i32(free), t)
        got = [x.tolist() for x in (t, p.q_off, p.lens, p.slots, p.positions)]
        assert got == [list(x) for x in want[:5]]
        assert p.taken.item() == want[5]
    assert p.status() == 0


@pytest.mark.parametrize("n,most", [(1, 5), (70, 900), (2500, 40)])
def test_plan_grows_its_lengths_in_place(cuda_device, n, most):
    """lens passed as cached, by one CTA and by many: the same plan, step by step."""
    torch, ref, nys = _mods()
    g = torch.Generator().manual_seed(n)
    page, steps = 16, 3
    fresh = [torch.randint(0, most + 1, (n,), generator=g).tolist() for _ in range(steps)]
    total = [sum(f) for f in fresh]
    width = max(sum(f) for f in zip(*fresh)) // page + 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    free = list(range(n * width))
    cached, table = [0] * n, [[-1] * width for _ in range(n)]
    t, lens = i32(table), i32(cached)
    for f, k in zip(fresh, total):
        p = nys.PagePlan(n, width, k, page, device=cuda_device)
        p.lens.copy_(lens)
        p.update(p.lens, i32(f), i32(free), t)
        table, off, cached, slots, positions, taken = ref.plan(cached, f, free, table, page)
        free, lens = free[taken:], p.lens
        got = [x.tolist() for x in (t, p.q_off, p.lens, p.slots, p.positions)]
        assert got == [table, off, cached, slots, positions]
        assert p.taken.item() == taken and p.status() == 0


def test_plan_without_pages_or_columns(cuda_device):
    torch, ref, nys = _mods()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cached, fresh, free, table = [3, 0, 4], [9, 10, 1], [9, 5, 7], [[2, -1, -1], [-1] * 3, [4, -1, -1]]
    t = i32(table)
    p = nys.PagePlan(3, 3, 20, 4, device=cuda_device)
    p.update(i32(cached), i32(fresh), i32(free), t)
    want = ref.plan(cached, fresh, free, table, 4)
    assert t.tolist() == want[0] and p.slots.tolist() == want[3] and p.taken.item() == 3
    assert p.status() == nys.NYS_PLAN_NO_PAGES
    p.clear_status()
    # A table that is too narrow.
    t2 = i32([[2], [-1], [4]])
    p2 = nys.PagePlan(3, 1, 20, 4, device=cuda_device)
    p2.update(i32(cached), i32(fresh), i32(list(range(10, 30))), t2)
    want = ref.plan(cached, fresh, list(range(10, 30)), [[2], [-1], [4]], 4)
    assert t2.tolist() == want[0] and p2.slots.tolist() == want[3]
    assert p2.status() == nys.NYS_PLAN_TABLE_FULL
    # Lengths that are negative or sum to less than the slots there are.
    p3 = nys.PagePlan(2, 4, 6, 4, device=cuda_device)
    t3 = i32([[-1] * 4] * 2)
    p3.update(i32([0, 0]), i32([-2, 3]), i32([1, 2, 3]), t3)
    assert p3.slots.tolist() == [4, 5, 6, -1, -1, -1] and p3.positions.tolist() == [0, 1, 2, -1, -1, -1]
    assert p3.status() == nys.NYS_PLAN_BAD_LENGTH


@pytest.mark.parametrize("fresh", [
    [2**31 - 1, 1, 5],           # the sum passes 31 bits
    [2**31 - 1, 2**31 - 1, 8],   # and 32 bits, to 6 = the slots there are
    [3, 2**31 - 1, 2**31 - 1, 5],
])
def test_plan_lengths_that_sum_past_32_bits(cuda_device, fresh):
    """Their sum is held, no other memory is reached, and the call is reported."""
    torch, _, nys = _mods()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    n, width, total = len(fresh), 4, 6
    plan = nys.PagePlan(n, width, total, 4, device=cuda_device)
    whole = torch.full((n + 2, width), -1, dtype=torch.int32, device=cuda_device)
    plan.update(i32([0] * n), i32(fresh), i32([9, 5, 7]), whole[1:n + 1])
    cell, want, row = iter([9, 5, 7]), [[-1] * width for _ in range(n + 2)], []
    for t in range(total):
        i = max(x for x in range(n) if sum(fresh[:x]) <= t)
        pos = t - sum(fresh[:i])
        if pos % 4 == 0:
            want[i + 1][pos // 4] = next(cell)
        row.append(want[i + 1][pos // 4] * 4 + pos % 4)
    assert whole.tolist() == want and plan.slots.tolist() == row
    assert plan.q_off.tolist() == [min(sum(fresh[:x]), total + 1) for x in range(n + 1)]
    assert plan.status() & nys.NYS_PLAN_BAD_LENGTH and plan.taken.item() == 3


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,kv,d,dv", [(1, 1, 64, 64), (64, 8, 128, 128), (333, 2, 20, 12),
                                            (50, 3, 4, 8), (5000, 4, 128, 64)])
@pytest.mark.parametrize("odd", [False, True])
def test_write(cuda_device, dtype, tokens, kv, d, dv, odd):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    page, n_pages = 16, tokens // 16 + 4
    pk = torch.randn((n_pages, page, kv, d), device=cuda_device).to(dt)
    pv = torch.randn((n_pages, page, kv, dv), device=cuda_device).to(dt)
    both = torch.randn((tokens, kv, d + dv + (1 if odd else 0)), device=cuda_device).to(dt)
    k, v = both[..., :d], both[..., -dv:]
    slots = torch.randperm(n_pages * page, device=cuda_device)[:tokens].contiguous()
    slots[::7] = -1
    slots[3::11] = n_pages * page
    wk, wv = pk.clone().view(-1, kv, d), pv.clone().view(-1, kv, dv)
    ok = (slots >= 0) & (slots < n_pages * page)
    wk[slots[ok]], wv[slots[ok]] = k[ok], v[ok]
    cache = nys.PagedKV(n_pages, page, kv, d, dv, dtype=dt, device=cuda_device, k=pk, v=pv)
    cache.write(k, v, slots)
    assert torch.equal(pk.view(-1, kv, d), wk) and torch.equal(pv.view(-1, kv, dv), wv)


# ------------------------------------------------- the tiled kernels' own corners
@pytest.mark.parametrize("dtype,q_lens,k_lens", [
    ("float32", [1300], [2350]), ("float32", [70, 1250], [1100, 1400]),
    ("bfloat16", [2500], [2500]), ("float16", [1, 2440], [1200, 2900])])
def test_prompt_last_round_is_cut(cuda_device, dtype, q_lens, k_lens):
    """Slightly more units than SMs: the rest's keys are cut into pieces and
    joined; values that are not finite still reach the rows that see them, and
    only those."""
    torch, ref, nys = _mods()
    _run_prompt(cuda_device, dtype, (16, 8, 128, 128), q_lens, k_lens)
    dt = getattr(torch, dtype)
    q, k, v, qo, ko = _inputs(torch, cuda_device, q_lens, k_lens, 16, 8, 128, 128, dt)
    want, wl, b, lb = ref.prompt(q, k, v, q_lens, k_lens, 2, 1 / math.sqrt(128), dt)
    at = sum(k_lens) - 40          # in the last sequence, seen by its last 40 queries
    v[at, 3, 9] = math.inf
    v[sum(k_lens[:-1]) + 5, 6, 1] = math.nan
    att = nys.ExactAttention(16, 8, 128, 128, dtype=dt, device=cuda_device)
    out = torch.empty_like(q)
    att.prompt(q, k, v, qo, out, k_off=ko)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[-40:, 6:8, 9] = True
    # Key 5 is seen from query 5 - (nk - nq) of its sequence on.
    hit[sum(q_lens[:-1]) + max(0, 5 - (k_lens[-1] - q_lens[-1])):, 12:14, 1] = True
    got = out.float().cpu()
    assert not torch.isfinite(got[hit]).any()
    ref.check(got[~hit], want[~hit], b[~hit], "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("geo,q_lens,k_lens", [
    ((16, 8, 128, 128), [1], [4001]), ((1, 1, 64, 64), [1], [30000]), ((1, 1, 64, 64), [1], [1600]),
    ((8, 1, 64, 128), [3, 1], [5000, 2]), ((16, 8, 128, 128), [16, 0, 2], [9000, 3000, 1]),
    ((4, 2, 64, 64), [130], [4000])])
def test_prompt_few_rows_of_many_keys(cuda_device, dtype, geo, q_lens, k_lens):
    """Fewer units than CTAs: every unit is cut."""
    _run_prompt(cuda_device, dtype, geo, q_lens, k_lens)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_without_workspace(cuda_device, dtype):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    lens = [200, 65] * 12
    q, k, v, qo, ko = _inputs(torch, cuda_device, lens, lens, 16, 8, 64, 64, dt)
    out = torch.empty_like(q)
    cfg = nys.NysAttnConfig(16, 8, 64, 64, nys._dtype_code(dt), 0.0)
    r = lambda t, h: nys._rows(t, dt, h, 64, "t")
    nys.nys_attn_prompt(cfg, len(lens), sum(lens), sum(lens), qo.data_ptr(), None, r(q, 16), r(k, 8),
                        r(v, 8), r(out, 16), stream=torch.cuda.current_stream().cuda_stream)
    want, _, b, _ = ref.prompt(q, k, v, lens, lens, 2, 1 / 8.0, dt)
    ref.check(out, want, b, "out")


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_row_offsets_past_32_bits(cuda_device, dtype):
    """Keys whose rows lie 2^24 elements apart: the last ones begin past 2^32."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    n, d, gap = 300, 64, 1 << 24
    q, k, v, qo, ko = _inputs(torch, cuda_device, [n], [n], 2, 1, d, d, dt)
    big = torch.empty(n * gap // (1 if dt != torch.float32 else 2), dtype=dt, device=cuda_device)
    step = big.numel() // n
    kk = big.as_strided((n, 1, d), (step, d, 1))
    vv = big.as_strided((n, 1, d), (step, d, 1), 4096)
    kk.copy_(k), vv.copy_(v)
    att = nys.ExactAttention(2, 1, d, d, dtype=dt, device=cuda_device)
    out = torch.empty_like(q)
    att.prompt(q, kk, vv, qo, out)
    want, _, b, _ = ref.prompt(q, k, v, [n], [n], 2, 1 / 8.0, dt)
    ref.check(out, want, b, "out")


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_result_does_not_depend_on_the_batch(cuda_device, dtype):
    """A sequence alone and in a large batch: within both results' bounds."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    lens = [77] + [(i * 29) % 190 for i in range(300)]
    q, k, v, qo, ko = _inputs(torch, cuda_device, lens, lens, 4, 2, 128, 128, dt)
    att = nys.ExactAttention(4, 2, 128, 128, dtype=dt, device=cuda_device)
    out = torch.empty_like(q)
    att.prompt(q, k, v, qo, out)
    alone = torch.empty_like(q[:77])
    att.prompt(q[:77], k[:77], v[:77], qo[:2].contiguous(), alone)
    want, _, b, _ = ref.prompt(q[:77], k[:77], v[:77], [77], [77], 2, 1 / math.sqrt(128), dt)
    ref.check(out[:77], want, b, "in the batch")
    ref.check(alone, want, b, "alone")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("geo", [(16, 8, 128, 128), (64, 1, 64, 64), (40, 1, 64, 128)])
def test_shared_wide_groups_and_long_prefix(cuda_device, dtype, geo):
    _run_shared(cuda_device, dtype, geo, [200, 3, 0, 66], 1500, 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_bad_value_in_the_prefix(cuda_device, dtype):
    """Infinities and NaN of the prefix and of own pages reach the requests that
    see them, in their channel."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, page, prefix, lens = 4, 2, 64, 16, 250, [20, 0, 33]
    k, v, pp, table = _pool(torch, cuda_device, lens, prefix, page, kv, d, d, dt)
    q = torch.randn((3, heads, d), device=cuda_device).to(dt)
    want, _, b, _ = ref.shared(q, k, v, pp, prefix, lens, table, 2, 1 / 8.0, dt)
    v[pp[1], 3, 0, 5] = math.inf       # the prefix, KV head 0
    v[table[2][1], 2, 1, 7] = math.nan  # request 2, KV head 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cache = nys.PagedKV(k.shape[0], page, kv, d, d, dtype=dt, device=cuda_device, k=k, v=v)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out = torch.empty((3, heads, d), device=cuda_device, dtype=dt)
    att.shared(q, cache, i32(lens), i32(table), out, prefix_pages=i32(pp), prefix_len=prefix)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[:, :2, 5] = True
    hit[2, 2:, 7] = True
    got = out.float().cpu()
    assert not torch.isfinite(got[hit]).any()
    ref.check(got[~hit], want[~hit], b[~hit], "out")


# A prefix is read by each request for itself while that is little, and else once
# by the tile kernel: the tests below have enough requests, or prefix, for that.
MANY = [(i * 7) % 5 for i in range(300)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("geo", GEOMETRIES)
def test_shared_prefix_read_once(cuda_device, dtype, geo):
    _run_shared(cuda_device, dtype, geo, MANY, 333, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix,page", [(40, 16), (128, 64), (127, 24), (300, 8), (129, 128),
                                         (1000, 7)])
def test_shared_prefix_read_once_lengths(cuda_device, dtype, prefix, page):
    _run_shared(cuda_device, dtype, (16, 8, 128, 128), MANY, prefix, page)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("geo,prefix", [((16, 8, 128, 128), 2600), ((64, 1, 64, 64), 5200),
                                        ((40, 1, 64, 128), 6800)])
def test_shared_prefix_read_once_by_few(cuda_device, dtype, geo, prefix):
    """Its tiles are dealt out over all CTAs."""
    _run_shared(cuda_device, dtype, geo, [200, 3, 0, 66], prefix, 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_prefix_read_once_bad_values_and_pages(cuda_device, dtype):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, page, prefix = 16, 8, 64, 16, 250
    k, v, pp, table = _pool(torch, cuda_device, MANY, prefix, page, kv, d, d, dt, junk=0.0)
    q = torch.randn((len(MANY), heads, d), device=cuda_device).to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cache = nys.PagedKV(k.shape[0], page, kv, d, d, dtype=dt, device=cuda_device, k=k, v=v)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out = torch.empty((len(MANY), heads, d), device=cuda_device, dtype=dt)
    run = lambda: att.shared(q, cache, i32(MANY), i32(table), out, prefix_pages=i32(pp),
                             prefix_len=prefix)
    want, _, b, _ = ref.shared(q, k, v, pp, prefix, MANY, table, 2, 1 / 8.0, dt)
    for bad in (math.inf, math.nan):
        kept = v[pp[1], 3, 0, 5].clone()
        v[pp[1], 3, 0, 5] = bad            # KV head 0, every request
        run()
        hit = torch.zeros(out.shape, dtype=torch.bool)
        hit[:, :2, 5] = True
        got = out.float().cpu()
        assert not torch.isfinite(got[hit]).any()
        ref.check(got[~hit], want[~hit], b[~hit], "out")
        v[pp[1], 3, 0, 5] = kept
    assert att.status() == 0
    pp[1], pp[4] = k.shape[0], -1
    run()
    want, _, b, _ = ref.shared(q, k, v, pp, prefix, MANY, table, 2, 1 / 8.0, dt)
    ref.check(out, want, b, "bad pages")
    assert att.status() == nys.NYS_ATTN_BAD_PAGE
    att.clear_status()


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_pieces_of_uneven_requests(cuda_device, dtype):
    """Few and many pieces a request in one call, with and without a prefix."""
    for lens, prefix in (([4000, 1, 0, 129, 700], 0), ([2500, 0, 31], 77), ([600] * 40 + [0, 1], 0)):
        _run_shared(cuda_device, dtype, (16, 8, 64, 64), lens, prefix, 32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("geo", [(16, 8, 128, 128), (1, 1, 64, 64), (20, 1, 64, 128), (6, 2, 96, 64)])
@pytest.mark.parametrize("lens,prefix", [([257, 1, 0], 0), ([900, 0, 129], 100), ([0, 0], 300),
                                         ([5000], 0), ([2000, 3], 0)])
def test_shared_pieces_that_join_in_a_cluster(cuda_device, dtype, geo, lens, prefix):
    """Two to eight pieces a request, some of them empty, and next to it more."""
    _run_shared(cuda_device, dtype, geo, lens, prefix, 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_cluster_bad_values(cuda_device, dtype):
    """A NaN or infinity in one piece reaches its request and channel, no other."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, page, lens = 4, 2, 64, 16, [700, 0, 300]
    k, v, _, table = _pool(torch, cuda_device, lens, 0, page, kv, d, d, dt)
    q = torch.randn((3, heads, d), device=cuda_device).to(dt)
    want, _, b, _ = ref.shared(q, k, v, [], 0, lens, table, 2, 1 / 8.0, dt)
    v[table[0][25], 3, 0, 5] = math.inf
    v[table[2][1], 2, 1, 7] = math.nan
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cache = nys.PagedKV(k.shape[0], page, kv, d, d, dtype=dt, device=cuda_device, k=k, v=v)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out = torch.empty((3, heads, d), device=cuda_device, dtype=dt)
    att.shared(q, cache, i32(lens), i32(table), out)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[0, :2, 5] = True
    hit[2, 2:, 7] = True
    got = out.float().cpu()
    assert not torch.isfinite(got[hit]).any()
    ref.check(got[~hit], want[~hit], b[~hit], "out")
    again = torch.empty_like(out)
    att.shared(q, cache, i32(lens), i32(table), again)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_prefix_read_once_in_a_graph(cuda_device, dtype):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, page, prefix = 16, 8, 128, 16, 300
    k, v, pp, table = _pool(torch, cuda_device, MANY, prefix, page, kv, d, d, dt, junk=0.0)
    q = torch.randn((len(MANY), heads, d), device=cuda_device).to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    tl, tt, tp = i32(MANY), i32(table), i32(pp)
    cache = nys.PagedKV(k.shape[0], page, kv, d, d, dtype=dt, device=cuda_device, k=k, v=v)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out = torch.empty_like(q)
    run = lambda: att.shared(q, cache, tl, tt, out, prefix_pages=tp, prefix_len=prefix)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    q.copy_(torch.randn_like(q))
    lens = [max(x - 1, 0) for x in MANY]
    tl.copy_(i32(lens))
    out.zero_()
    graph.replay()
    want, _, b, _ = ref.shared(q, k, v, pp, prefix, lens, table, 2, 1 / math.sqrt(d), dt)
    ref.check(out, want, b, "replayed")
    assert att.status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_in_a_graph(cuda_device, dtype):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, page, prefix, lens = 8, 2, 128, 16, 300, [40, 500, 1]
    k, v, pp, table = _pool(torch, cuda_device, lens, prefix, page, kv, d, d, dt, junk=0.0)
    q = torch.randn((3, heads, d), device=cuda_device).to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    tl, tt, tp = i32(lens), i32(table), i32(pp)
    cache = nys.PagedKV(k.shape[0], page, kv, d, d, dtype=dt, device=cuda_device, k=k, v=v)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    out = torch.empty_like(q)
    run = lambda: att.shared(q, cache, tl, tt, out, prefix_pages=tp, prefix_len=prefix)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    q.copy_(torch.randn_like(q))
    tl.copy_(i32([33, 499, 0]))
    out.zero_()
    graph.replay()
    want, _, b, _ = ref.shared(q, k, v, pp, prefix, [33, 499, 0], table, 4, 1 / math.sqrt(d), dt)
    ref.check(out, want, b, "replayed")


@pytest.mark.parametrize("dtype", TYPES)
def test_graph_keeps_its_workspace(cuda_device, dtype):
    """A larger call after a capture takes a new workspace; the graph's stays."""
    torch, _, nys = _mods()
    dt = getattr(torch, dtype)
    att = nys.ExactAttention(8, 2, 64, 64, dtype=dt, device=cuda_device)
    torch.manual_seed(5)

    def args(lens):
        off = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32,
                           device=cuda_device)
        rows = sum(lens)
        make = lambda h: torch.randn((rows, h, 64), device=cuda_device).to(dt)
        return make(8), make(2), make(2), off, torch.zeros((rows, 8, 64), device=cuda_device, dtype=dt)

    # f32 holds its keys' pieces there; 16-bit types a counter, and for few long
    # prompts pieces of results.
    small, large = args([2000] if dtype == "float32" else [1000] * 20), args([6000, 100])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        att.prompt(*small)
        want = small[4].clone()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            att.prompt(*small)
        before = att._work_ptr
        att.prompt(*large)
        assert att._work_ptr != before
        # Had the graph's workspace been freed, these would lie in it.
        others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device=cuda_device) for _ in range(64)]
        small[4].zero_()
        graph.replay()
        side.synchronize()
    assert torch.equal(small[4], want)
    assert all(bool((x == 7).all()) for x in others)
    assert att.status() == 0


def test_workspace_is_asked_for_again_after_it_was_refused(cuda_device, monkeypatch):
    """An allocation that failed leaves no note of its size behind: the same call
    made again takes the workspace then, and the tiled kernel."""
    torch, ref, nys = _mods()
    q, k, v, qo, ko = _inputs(torch, cuda_device, [300], [300], 4, 2, 64, 64, torch.float32)
    att = nys.ExactAttention(4, 2, 64, 64, device=cuda_device)
    out = torch.empty_like(q)

    def refuse(*a, **kw):
        raise torch.cuda.OutOfMemoryError("out of memory")
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", refuse)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            att.prompt(q, k, v, qo, out)
    att.prompt(q, k, v, qo, out)
    assert att._work_bytes >= nys.nys_attn_workspace_bytes(att.cfg, 1, 300, 300) > 0
    want, _, b, _ = ref.prompt(q, k, v, [300], [300], 2, 1 / 8.0, torch.float32)
    ref.check(out, want, b, "out")


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_units_of_every_kind_in_any_order(cuda_device, dtype):
    """Units of one and two query tiles, with one, many and no key tiles, follow
    each other in every order on a CTA: no barrier may run a phase ahead of who
    waits on it.  Every launch gives the same bits and none gives up."""
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(11)
    att = nys.ExactAttention(4, 2, 64, 64, dtype=dt, device=cuda_device)
    for n, top, more in ((700, 28, 300), (400, 150, 0), (300, 70, 900), (64, 300, 0)):
        q_lens = torch.randint(0, top, (n,), generator=g).tolist()
        # Some sequences' first queries see no key at all, some see many.
        k_lens = [max(0, x - 20) if i % 3 == 0 else x + (more if i % 5 == 0 else 0)
                  for i, x in enumerate(q_lens)]
        q, k, v, qo, ko = _inputs(torch, cuda_device, q_lens, k_lens, 4, 2, 64, 64, dt)
        first = torch.empty_like(q)
        att.prompt(q, k, v, qo, first, k_off=ko)
        again = torch.empty_like(q)
        for _ in range(150):
            again.zero_()
            att.prompt(q, k, v, qo, again, k_off=ko)
            assert torch.equal(first, again)
        assert att.status() == 0
