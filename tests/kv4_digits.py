"""How many digits f32 results of attention over the 4-bit cache have, and what a kernel
with fewer would give: kv4_reference.attend's bound holds every single number in the worst
case, and would let a weight of 11 bits pass."""
import math

import torch

# |result - exact| / |exact| of a call's heads, as norms.  Keys whose values have nothing in
# common: a result and its error are both sums of independent parts, so this is a weight's
# error, relative, on average.  Weights in two f16 pieces 2^-22, the exponential 2^-22 and
# its argument, rounded at up to 16, 2^-21: half of that on average, 2^-21 together.
# Scores: sums of d / 16 products and pieces of sums of about 1, each cut off by up to 2^-23
# (half that on average): 32 * 2^-24 * 1 = 2^-19 for d = 256 if all went one way.  Queries
# 2^-22 of the row.  2^-18 is twice their sum; one f16 piece of a weight is off by 2^-12
# at most, 2^-13 on average.
MOST = 2.0 ** -18


def off(got, want):
    return float((got - want).norm() / want.norm())


def attend(q, k, v, scale, piece):
    """Attention in float64 but for the weights: each key's p * step is rounded as `piece`
    does, group by group.  q [heads][d]; k [t][kv][d]; v a (codes, steps, middles) triple."""
    codes, steps, mids = v
    group = q.shape[0] // k.shape[1]
    each = lambda x: x.double().repeat_interleave(group, 1)  # noqa: E731
    s = torch.einsum("hd,thd->ht", q.double(), each(k)) * scale
    p = torch.exp(s - s.amax(-1, keepdim=True))
    spread = lambda x: x.repeat_interleave(64, -1)[..., :codes.shape[-1]]  # noqa: E731
    weights = piece(p.t()[:, :, None] * each(steps))           # [t][heads][groups]
    out = (spread(weights) * (each(codes) - 8)).sum(0) + (p.t()[:, :, None] * spread(each(mids))).sum(0)
    return out / p.sum(-1, keepdim=True)


def one_f16(x):
    """The first piece alone, at the size that fits the largest (a power of two)."""
    up = 2.0 ** (14 - math.floor(math.log2(float(x.max()))))
    return (x * up).to(torch.float16).double() / up


def bf16(x):
    return x.to(torch.bfloat16).double()


def two_f16(x):
    up = 2.0 ** (14 - math.floor(math.log2(float(x.max()))))
    y = x * up
    first = y.to(torch.float16).double()
    return (first + (y - first).to(torch.float16).double()) / up
