"""Plain forms, in 64 bits or number by number, of norm and rotation and of the
4-bit cache (include/nys.h), and the bounds their kernels are held to."""
import math

import torch

U = 2.0 ** -24                       # a rounding of f32, relative
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def turned(x, weight, eps, positions, freqs, interleaved, shift=0):
    """Norm and rotation of [rows][heads][d] in float64, and the size (|a| + |b| of a
    number's pair) that its error goes by."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
    y, size = x.clone(), x.abs()
    half = len(freqs)
    if half:
        f = torch.tensor(freqs, dtype=torch.float64, device=x.device)
        t = ((positions.double() + shift)[:, None] * f)[:, None]
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
        y[..., b] = x[..., a] * t.sin() + x[..., b] * t.cos()
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def turned_bound(want, size, dtype, far=0):
    """A sum of up to 256 squares lies over 32 lanes: 8 products and 5 sums of lanes, 14
    roundings with the division by d, halved by the root; the reciprocal root 2 units in
    the last place (4 U), two factors: 13 U.  The turn is rounded to 24 bits (a half-turn
    of 2^-25: pi / 2 U), sine and cosine are off by 2 U, two products and a sum: 7 U more.
    The plain form's own angle is off by far * 2^-53."""
    return 20 * U * size + far * 2.0 ** -53 * size + EPS[dtype] * (want.abs() + 20 * U * size) + TINY[dtype]


def quantize(x):
    """Codes [..][d] (int64), steps and middles [..][groups] of f32 rows, operation by
    operation as nys.h gives them (numpy rounds each to f32, quotients correctly)."""
    import numpy as np
    x = x.float().cpu().numpy()
    f, d = np.float32, x.shape[-1]
    codes = np.zeros(x.shape, np.int64)
    steps, mids = [], []
    with np.errstate(all="ignore"):
        for at in range(0, d, 64):
            part = x[..., at:at + 64]
            lo, hi = part.min(-1, keepdims=True), part.max(-1, keepdims=True)
            bf = lambda z: torch.from_numpy(np.ascontiguousarray(z)).bfloat16().float().numpy()  # noqa: E731
            mid = bf(lo + (hi - lo) * f(8) / f(15))
            step = np.maximum((hi - mid) / f(7), (mid - lo) * f(0.125))
            low = bf(step)           # to the nearest; the next one up where that is below
            up = (np.ascontiguousarray(low).view(np.uint32) + np.uint32(0x10000)).view(f)
            step = np.where(low < step, up, low)
            bad = ~(np.isfinite(part).all(-1, keepdims=True) & np.isfinite(mid) & np.isfinite(step))
            step = np.where(step < f(2.0 ** -100), f(0), step)
            flat = bad | (step == 0)
            c = np.rint((part - mid) / np.where(flat, f(1), step))
            codes[..., at:at + 64] = np.where(flat, 8, np.clip(np.where(flat, 0, c), -8, 7) + 8)
            steps.append(np.where(bad, f(np.nan), step))
            mids.append(np.where(bad, f(np.nan), mid))
    return (torch.from_numpy(codes), torch.from_numpy(np.concatenate(steps, -1)),
            torch.from_numpy(np.concatenate(mids, -1)))


def unpack(data, kv_heads, d, dv, page):
    """A cache's codes [slots][kv_heads][d], steps and middles [slots][kv_heads][groups],
    of keys and of values, number by number from the block's words."""
    data = data.cpu().contiguous()
    pages = data.shape[0]
    G = -(-max(d, dv) // 64)
    words = data.view(-1).view(torch.int32).long() & 0xffffffff
    words = words.view(pages, kv_heads, page // 16, 288 * G)
    slot = torch.arange(pages * page)
    pg, block, t = slot // page, slot % page // 16, slot % 16
    place = t % 8 // 2 * 4 + t // 8 * 2 + t % 2
    out = []
    for values, dim in ((False, d), (True, dv)):
        x = torch.arange(dim)
        g, e = x // 64, x % 64
        if values:
            word = 128 * G + (g * 128 + e // 8 * 16)[None] + place[:, None]
        else:
            word = (g * 128 + e % 32 // 8 * 4 + e // 32)[None] + (t % 8 * 16 + t // 8 * 2)[:, None]
        at = words[pg, :, block]                                     # [slots][kv][words]
        codes = torch.gather(at, 2, word[:, None].expand(-1, kv_heads, -1)) >> (4 * (e % 8)) & 15
        word = (272 if values else 256) * G + (torch.arange(-(-dim // 64)) * 16)[None] + place[:, None]
        scale = torch.gather(at, 2, word[:, None].expand(-1, kv_heads, -1))
        f = lambda b: (b << 16).to(torch.uint32).view(torch.float32)  # noqa: E731
        out.append((codes, f(scale >> 16), f(scale & 0xffff)))
    return out


def values(codes, step, mid):
    """What they stand for, in float64 (exact)."""
    d = codes.shape[-1]
    spread = lambda z: z.double().repeat_interleave(64, -1)[..., :d]  # noqa: E731
    return spread(mid) + spread(step) * (codes - 8)


def attend(q, k, v, scale, dtype):
    """One token: q [heads][d] over k [t][kv_heads][d], v [t][kv_heads][dv] in float64: the
    result, its log-sum and the result's bound."""
    heads, kv = q.shape[0], k.shape[1]
    q, k, v = (x.double().cpu() for x in (q, k, v))
    group = heads // kv
    if not len(k):
        z = torch.zeros(heads, v.shape[2], dtype=torch.float64)
        return z, torch.full((heads,), -math.inf, dtype=torch.float64), z + TINY[dtype]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    s = torch.einsum("hd,thd->ht", q, k) * scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    out = torch.einsum("ht,thd->hd", p, v)
    size = torch.einsum("ht,thd->hd", p, v.abs())
    return out, lse, attend_bound(q, k, s, p, out, size, v, scale, dtype)


def attend_bound(q, k, s, p, out, size, v, scale, dtype):
    """Scores: queries to 22 bits, products of d numbers summed by the matrix unit, which
    may cut each of the d / 16 + 4 partial sums at 2^-23 of what is summed, and a code's 8
    may be added to either sign of it; the exponent is rounded at the score's size.  That
    is an error of a weight, relative.  Weights: 16 bits (f32: 24), the exponential 2^-21.
    Sums: one cut of 2^-23 a product of 16 keys and piece; a group's values reach from
    -8 to 7 steps around its middle, of which |v| may be small: those steps count."""
    terms = torch.einsum("hd,thd->ht", q.abs(), k.abs()).amax(-1) * scale
    spread = q.abs().sum(-1) * (k.amax((0, 2)) - k.amin((0, 2))) * scale
    score = (2.0 ** -22 + (q.shape[1] / 16 + 4) * 2.0 ** -23) * (terms + spread) + 2 * U * (s.abs().amax(-1) + 32)
    keys = s.shape[1]
    weight = 2.0 ** -21 + (2.0 ** -22 if dtype == torch.float32 else 2.0 ** -16)
    sums = 3 * (keys / 16 + 8) * 2.0 ** -23
    reach = size + (v.amax((0, 2)) - v.amin((0, 2)))[:, None]
    rel = 2 * (score + weight + sums)[:, None]
    return rel * reach + EPS[dtype] * (out.abs() + rel * reach) + TINY[dtype]


def lse_bound(q, k, scale, lse):
    """Scores as above, sums of at most 2^20 weights in order of lanes and blocks."""
    q, k = q.double().cpu(), k.double().cpu()
    k = k.repeat_interleave(q.shape[0] // k.shape[1], 1)
    terms = torch.einsum("hd,thd->ht", q.abs(), k.abs()).amax(-1) * scale
    spread = q.abs().sum(-1) * (k.amax((0, 2)) - k.amin((0, 2))) * scale
    return ((2.0 ** -22 + (q.shape[1] / 16 + 4) * 2.0 ** -23) * (terms + spread)
            + (k.shape[0] / 64 + 16) * U + 2 * U * (lse.abs() + 64))


def check(got, want, bound, where):
    got = got.double().cpu()
    want, bound = want.cpu(), bound.cpu()
    wrong = ~((got - want).abs() <= bound)
    assert not bool(wrong.any()), (
        f"{where}: {int(wrong.sum())} of {wrong.numel()} off, worst "
        f"{float(((got - want).abs() / bound).max()):.2f} of the bound")
