"""Plain 64-bit forms of the exact-attention operators on the CPU, with an
error bound for every output element, for the tests."""
import math

import torch

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend(q, k, v, seen, scale, dtype):
    """One head: q [r][d], k [t][d], v [t][dv] float64, seen [r][t] bool.
    Returns out, lse and a bound on each one's error.

    The bound counts roundings.  A score is a dot product of d terms summed in
    f32, each product good to 2^-21 (fp32 operands may be taken as pairs of
    16-bit pieces): |ds| <= (2^-21 + d 2^-24) scale sum_c |q_c k_c|.  A weight
    e^{s - m} then is off by 2 |ds| relative (its own score and the maximum's
    share), 2^-20 for the exponential and its argument's rounding (arguments
    count |s - m| 2^-23), and half a step of the stored type where the weights
    are rounded for the second product (16-bit types).  Sums of t terms add
    t 2^-24.  Numerator and denominator each carry it, and the result is
    rounded once more to its type."""
    r, t = seen.shape
    s = (q @ k.T) * scale
    s = s.masked_fill(~seen, -math.inf)
    mag = (q.abs() @ k.abs().T) * scale
    ds = (mag.masked_fill(~seen, 0.0).amax(dim=1) if t else q.new_zeros(r)) * (
        2.0 ** -21 + q.shape[1] * 2.0 ** -24)
    m = s.amax(dim=1) if t else q.new_full((r,), -math.inf)
    ref = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - ref[:, None])
    p = p.masked_fill(~seen, 0.0)
    total = p.sum(dim=1)
    safe = torch.where(total == 0, torch.ones_like(total), total)
    w = p / safe[:, None]
    vz = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    out = w @ vz
    low = torch.where(seen & (p > 2.0 ** -60), ref[:, None] - s, torch.zeros_like(s))
    arg = (low.amax(dim=1) if t else q.new_zeros(r)) * 2.0 ** -23
    rel = 2 * ds + arg + 2.0 ** -20 + t * 2.0 ** -24
    half = 0.0 if dtype == torch.float32 else EPS[dtype]
    bound = (w @ vz.abs()) * (2 * rel + half)[:, None] + EPS[dtype] * out.abs() * (1 + 2 ** -6)
    bound = bound + (2.0 ** -24 if dtype == torch.float16 else 1e-37)   # its smallest step
    lse = torch.where(total == 0, torch.full_like(total, -math.inf), ref + torch.log(safe))
    lse_bound = rel + 2.0 ** -22 * (1 + ref.abs())
    return out, lse, bound, lse_bound


def check(got, want, bound, what):
    got, same = got.double().cpu(), torch.isinf(want)
    assert torch.equal(got[same], want[same]), f"{what}: infinities differ"
    err = (got[~same] - want[~same]).abs()
    assert bool(torch.isfinite(err).all()), f"{what}: not finite"
    bad = err > bound[~same]
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {err.numel()} outside, worst "
                                 f"{float((err / bound[~same]).max()):.2f} x its bound")


def prompt(q, k, v, q_lens, k_lens, group, scale, dtype):
    """Packed causal attention; q [rows][heads][d], k, v [keys][kv_heads][..]."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    heads = q.shape[1]
    out = torch.zeros((q.shape[0], heads, v.shape[2]), dtype=torch.float64)
    lse = torch.zeros((q.shape[0], heads), dtype=torch.float64)
    b, lb = torch.zeros_like(out), torch.zeros_like(lse)
    q0 = k0 = 0
    for nq, nk in zip(q_lens, k_lens):
        i, j = torch.arange(nq)[:, None], torch.arange(nk)[None, :]
        seen = j <= i + nk - nq
        for h in range(heads):
            g = h // group
            sl = slice(q0, q0 + nq)
            out[sl, h], lse[sl, h], b[sl, h], lb[sl, h] = attend(
                q[sl, h], k[k0:k0 + nk, g], v[k0:k0 + nk, g], seen, scale, dtype)
        q0, k0 = q0 + nq, k0 + nk
    return out, lse, b, lb


def shared(q, pool_k, pool_v, prefix_pages, prefix_len, lens, table, group, scale, dtype):
    """One token over a shared prefix and paged own keys; a page outside the
    pool counts as zeros."""
    q, pool_k, pool_v = q.double().cpu(), pool_k.double().cpu(), pool_v.double().cpu()
    n_pages, page = pool_k.shape[:2]
    heads = q.shape[1]

    def rows(pool, pages, count):
        parts = [pool[p] if 0 <= p < n_pages else torch.zeros_like(pool[0])
                 for p in pages[:-(-count // page)]]
        return torch.cat(parts)[:count] if parts else pool[:0].reshape(0, *pool.shape[2:])

    out = torch.zeros((q.shape[0], heads, pool_v.shape[3]), dtype=torch.float64)
    lse = torch.zeros((q.shape[0], heads), dtype=torch.float64)
    b, lb = torch.zeros_like(out), torch.zeros_like(lse)
    kp, vp = rows(pool_k, prefix_pages, prefix_len), rows(pool_v, prefix_pages, prefix_len)
    for i in range(q.shape[0]):
        k = torch.cat([kp, rows(pool_k, table[i], lens[i])])
        v = torch.cat([vp, rows(pool_v, table[i], lens[i])])
        seen = torch.ones((1, k.shape[0]), dtype=torch.bool)
        for h in range(heads):
            g = h // group
            r = attend(q[i, h][None], k[:, g], v[:, g], seen, scale, dtype)
            out[i, h], lse[i, h], b[i, h], lb[i, h] = r[0][0], r[1][0], r[2][0], r[3][0]
    return out, lse, b, lb


def plan(cached, fresh, free, table, page):
    """Block tables, offsets, lengths, slots, positions and pages taken."""
    table = [list(row) for row in table]
    q_off, slots, positions, at = [0], [], [], 0
    for i, (c, f) in enumerate(zip(cached, fresh)):
        old, new = -(-c // page), -(-(c + f) // page)
        for col in range(old, new):
            if col < len(table[i]):
                table[i][col] = free[at] if at < len(free) else -1
            at += 1
        for x in range(c, c + f):
            col = x // page
            pg = table[i][col] if col < len(table[i]) else -1
            slots.append(-1 if pg < 0 else pg * page + x % page)
            positions.append(x)
        q_off.append(q_off[-1] + f)
    return (table, q_off, [c + f for c, f in zip(cached, fresh)], slots, positions,
            min(at, len(free)))
