"""The operators between a layer's projections and its attention, and the cache
in 4 bits, as measured workloads: their inputs, their plain form and their
64-bit form.

  norm     RMS norms of queries and keys for each head, with the rotation by
           their positions
  append   the same, with the rotated keys and the values going into the pages
           of their slots
  write4   keys and values into a paged cache of 4 bits, and all its rows read
           back as the values they stand for
  attend4  one token of attention for each request over such a cache

``listed()`` gives the fixed cases, ``draw()`` more of the same ranges.  With
``own`` false ``run`` computes an operator in elementary torch operations,
with ``own`` true it makes the calls of streaming_nystr_landmark_gb300.nys.
Geometries are those of workloads.py: 16 query heads over 8 KV heads with
head dim 128 (``layer``, ``batch64``), 32 over 4 (``long``), 1 over 1 with
head dim 64 (``single``).

A 4-bit cache holds each row in groups of 64 numbers: a step and a middle in
bf16 and 64 codes, value = middle + step * (code - 8).  Its bytes are
[page][KV head][block of 16 tokens][1152 * groups], where a block is the keys'
codes, the values' codes, the keys' scales and the values' scales, in 32-bit
words:
  keys' codes    [group][token % 8][c][token / 8][h]      8 codes, from 64 group + 32 h + 8 c
  values' codes  [group][r][token % 8 / 2][token / 8][token % 2]  8 codes, from 64 group + 8 r
  scales         [group][token % 8 / 2][token / 8][token % 2]     step << 16 | middle
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def listed():
    wide = {"heads": 16, "kv_heads": 8, "d": 128, "rot": 128}
    long = {"heads": 32, "kv_heads": 4, "d": 128, "rot": 128}
    return [
        # One request's new token: a launch's latency.
        {"name": "norm token bf16", "op": "norm", "type": "bf16", **wide, "inter": False, "base": 1e6,
         "n": 1, "tokens": 1, "far": 4096},
        # The prompts of batch64's layers, in the framework's own type.
        {"name": "norm prompts f32", "op": "norm", "type": "f32", **wide, "inter": False, "base": 1e6,
         "n": 64, "tokens": 16384, "far": 1},
        # A part of a very long prompt at the long-context geometry: far positions.
        {"name": "norm long bf16", "op": "norm", "type": "bf16", **long, "inter": True, "base": 5e5,
         "n": 1, "tokens": 32768, "far": 1000000},
        # A decode step's rows: one token of each of 64 requests.
        {"name": "append decode bf16", "op": "append", "type": "bf16", **wide, "inter": False, "base": 1e6,
         "n": 64, "tokens": 64, "far": 4000, "page": 16},
        # Admission of 64 prompts.
        {"name": "append prompts f32", "op": "append", "type": "f32", **wide, "inter": False, "base": 1e6,
         "n": 64, "tokens": 16384, "far": 1, "page": 16},
        # Prompts of a geometry of odd sizes, a part of each head rotated, continued after what is cached.
        {"name": "append partial f16", "op": "append", "type": "f16", "heads": 14, "kv_heads": 2, "d": 80,
         "rot": 52, "inter": False, "base": 1e4, "n": 7, "tokens": 4099, "far": 3000, "page": 64},
        # A decode step's rows into the 4-bit cache.
        {"name": "write4 decode bf16", "op": "write4", "type": "bf16", "kv_heads": 8, "d": 128, "n": 64,
         "tokens": 64, "far": 4000, "page": 16},
        # A batch of prompts' rows.
        {"name": "write4 prompts bf16", "op": "write4", "type": "bf16", "kv_heads": 8, "d": 128, "n": 64,
         "tokens": 16384, "far": 1, "page": 64},
        # A handful of young requests: latency.
        {"name": "attend4 few bf16", "op": "attend4", "type": "bf16", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 4, "lo": 3, "hi": 345, "page": 16},
        # 64 chats in the framework's own type.
        {"name": "attend4 chats f32", "op": "attend4", "type": "f32", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 64, "lo": 97, "hi": 3025, "page": 16},
        # Many requests of any age, the cache's bytes being what counts.
        {"name": "attend4 batch bf16", "op": "attend4", "type": "bf16", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 128, "lo": 517, "hi": 8192, "page": 64},
        # Two very long requests at the long-context geometry.
        {"name": "attend4 long bf16", "op": "attend4", "type": "bf16", "heads": 32, "kv_heads": 4, "d": 128,
         "n": 2, "lo": 131075, "hi": 200000, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "append", "write4", "attend4", "attend4", "attend4"])
    kind = rng.choice(list(TYPES))
    heads, kv_heads = rng.choice([(16, 8), (32, 4), (1, 1), (8, 8), (12, 4), (14, 2), (24, 8)])
    d = rng.choice([64, 128, 128, 96, 80])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    if op == "attend4":
        n = _log(rng, 1, 200)
        hi = _log(rng, 1, min(100000, 400000 // n))
        return {"op": op, "type": kind, "heads": heads, "kv_heads": kv_heads, "d": d, "n": n,
                "lo": _log(rng, 1, hi), "hi": hi, "page": page}
    tokens = _log(rng, 1, 16384)
    n = _log(rng, 1, min(tokens, 256))
    c = {"op": op, "kv_heads": kv_heads, "d": d, "n": n, "tokens": tokens, "far": _log(rng, 1, 100000), "page": page}
    if op == "write4":
        return {**c, "type": rng.choice(["bf16", "f16"])}
    rot = rng.choice([d, d, d // 2, d // 2 + 12])
    return {**c, "type": kind, "heads": heads, "rot": rot, "inter": rng.random() < 0.4,
            "base": rng.choice([1e4, 5e5, 1e6])}


def _randn(gen, shape, kind):
    return torch.randn(shape, generator=gen, device=DEV).to(TYPES[kind])


def _keys(gen, rows, kv_heads, d):
    """Keys with a mean direction for each head, as workloads.py draws them."""
    u = torch.randn((1, kv_heads, d), generator=gen, device=DEV)
    return torch.randn((rows, kv_heads, d), generator=gen, device=DEV) + 2.0 * u / u.norm(dim=-1, keepdim=True)


def _frequencies(case):
    """Angle a position of each pair, in float64."""
    rot = case["rot"]
    return case["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    make = {"norm": _prepare_rows, "append": _prepare_rows, "write4": _prepare_write4, "attend4": _prepare_attend4}
    state = make[case["op"]](case, gen, np.random.RandomState(int(seed) % (1 << 31)))
    state["op"] = case["op"]
    return state


def _places(case, rs):
    """Positions and, where there are pages, slots of the batch's tokens: n requests of about the same number of new
    tokens, each continued from a position below `far`; its pages are anywhere in the pool."""
    n, tokens = case["n"], case["tokens"]
    # The same requests for every seed, in another order, so that the pool has as many pages.
    counts = np.full(n, tokens // n)
    counts[:tokens % n] += 1
    starts = np.random.RandomState(7).randint(0, case["far"], n)
    order = rs.permutation(n)
    counts, starts = counts[order], starts[order]
    request = np.repeat(np.arange(n), counts)
    at = np.arange(tokens) - np.repeat(np.cumsum(counts) - counts, counts)
    positions = starts[request] + at
    if "page" not in case:
        return torch.tensor(positions, dtype=torch.int32, device=DEV), None, 0
    page = case["page"]
    inner = starts % page  # only the pages that get tokens are here
    need = -(-(inner + counts) // page)
    pages = int(need.sum()) + 3
    order = rs.permutation(pages)
    first = np.cumsum(need) - need
    x = inner[request] + at
    slots = order[first[request] + x // page] * page + x % page
    return (torch.tensor(positions, dtype=torch.int32, device=DEV),
            torch.tensor(slots, dtype=torch.int64, device=DEV), pages)


def _prepare_rows(case, gen, rs):
    heads, kv, d, kind, tokens = case["heads"], case["kv_heads"], case["d"], case["type"], case["tokens"]
    # One projection's output: a token's queries, keys and values side by side.
    qkv = _randn(gen, (tokens, heads + 2 * kv, d), kind) * 1.5
    weights = [1 + 0.1 * torch.randn(d, generator=gen, device=DEV) for _ in range(2)]
    positions, slots, pages = _places(case, rs)
    s = {"q": qkv[:, :heads], "k": qkv[:, heads:heads + kv], "v": qkv[:, heads + kv:], "positions": positions,
         "slots": slots, "q_weight": weights[0], "k_weight": weights[1], "inter": case["inter"],
         "freqs": _frequencies(case).to(DEV), "rot": case["rot"],
         "q_out": torch.empty((tokens, heads, d), dtype=qkv.dtype, device=DEV),
         "k_out": torch.empty((tokens, kv, d), dtype=qkv.dtype, device=DEV)}
    if case["op"] == "append":
        page = case["page"]
        s["pool_k"] = _randn(gen, (pages, page, kv, d), kind)
        s["pool_v"] = _randn(gen, (pages, page, kv, d), kind)
    if own:
        from streaming_nystr_landmark_gb300 import nys
        rotation = nys.Rotation(d, base=case["base"], rot=case["rot"], interleaved=case["inter"], device=DEV)
        s["prepare"] = nys.QKPrepare(heads, kv, d, dtype=qkv.dtype, q_weight=weights[0], k_weight=weights[1], eps=EPS,
                                     rotation=rotation, device=DEV)
        if case["op"] == "append":
            s["cache"] = nys.PagedKV(pages, page, kv, d, d, dtype=qkv.dtype, device=DEV, k=s["pool_k"], v=s["pool_v"])
    return s


def _pool4(k, v, page):
    """The bytes of a 4-bit cache that holds these rows ([slots][kv_heads][d], f32)."""
    slots, kv, d = k.shape
    groups = -(-d // 64)
    blocks = torch.empty((slots // 16, kv, 288 * groups), dtype=torch.int32, device=DEV)
    t, c, h, r = 16, 4, 2, 8
    for x, codes_at, scales_at, is_k in ((k, 0, 256 * groups, True), (v, 128 * groups, 272 * groups, False)):
        codes, step, mid = _quantize(x)
        codes = torch.nn.functional.pad(codes, (0, 64 * groups - d), value=8).to(torch.int32)
        shifts = 4 * torch.arange(8, dtype=torch.int32, device=DEV)
        words = (codes.view(slots, kv, 8 * groups, 8) << shifts).sum(dim=-1, dtype=torch.int32)
        words = words.view(-1, t, kv, groups, 8)
        if is_k:  # [block][t8][t][kv][group][h][c] -> [block][kv][group][t][c][t8][h]
            words = words.view(-1, 2, 8, kv, groups, h, c).permute(0, 3, 4, 2, 6, 1, 5)
        else:  # [block][t8][t2][t1][kv][group][r] -> [block][kv][group][r][t2][t8][t1]
            words = words.view(-1, 2, 4, 2, kv, groups, r).permute(0, 4, 5, 6, 2, 1, 3)
        blocks[:, :, codes_at:codes_at + 128 * groups] = words.reshape(-1, kv, 128 * groups)
        scale = step.to(torch.bfloat16).view(torch.int16).int() << 16
        scale = scale | (mid.to(torch.bfloat16).view(torch.int16).int() & 0xffff)
        scale = scale.view(-1, 2, 4, 2, kv, groups).permute(0, 4, 5, 2, 1, 3)
        blocks[:, :, scales_at:scales_at + 16 * groups] = scale.reshape(-1, kv, 16 * groups)
    blocks = blocks.view(slots // page, page // 16, kv, -1).transpose(1, 2).contiguous()
    return blocks.view(torch.uint8).view(slots // page, kv, -1)


def _prepare_write4(case, gen, rs):
    kv, d, kind, page, tokens = case["kv_heads"], case["d"], case["type"], case["page"], case["tokens"]
    _, slots, pages = _places(case, rs)
    old = [_keys(gen, pages * page, kv, d), torch.randn((pages * page, kv, d), generator=gen, device=DEV)]
    s = {"k": _keys(gen, tokens, kv, d).to(TYPES[kind]), "v": _randn(gen, (tokens, kv, d), kind), "slots": slots,
         "data": _pool4(*old, page), "kv_heads": kv, "d": d, "page": page,
         "every": torch.arange(pages * page, dtype=torch.int64, device=DEV),
         "k_out": torch.empty((pages * page, kv, d), dtype=TYPES[kind], device=DEV),
         "v_out": torch.empty((pages * page, kv, d), dtype=TYPES[kind], device=DEV)}
    if own:
        from streaming_nystr_landmark_gb300 import nys
        s["cache"] = nys.PagedKV4(pages, page, kv, d, d, dtype=TYPES[kind], device=DEV, data=s["data"])
    return s


def _lengths(case):
    """The batch's lengths, spread geometrically from hi down to lo."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    return [int(round(hi * (lo / hi) ** (i / max(1, n - 1)))) for i in range(n)]


def _prepare_attend4(case, gen, rs):
    heads, kv, d, kind, page = case["heads"], case["kv_heads"], case["d"], case["type"], case["page"]
    lengths = rs.permutation(_lengths(case))
    need = -(-lengths // page)
    pages = int(need.sum()) + 3
    order = rs.permutation(pages).astype(np.int32)
    table = np.full((case["n"], max(need)), -1, dtype=np.int32)
    table[np.arange(max(need))[None, :] < need[:, None]] = order[:int(need.sum())]
    rows = pages * page
    s = {"q": _randn(gen, (case["n"], heads, d), kind),
         "data": _pool4(_keys(gen, rows, kv, d), torch.randn((rows, kv, d), generator=gen, device=DEV), page),
         "lens": torch.tensor(lengths.astype(np.int32), device=DEV), "table": torch.tensor(table, device=DEV),
         "kv_heads": kv, "page": page, "d": d}
    if own:
        from streaming_nystr_landmark_gb300 import nys
        s["attention"] = nys.ExactAttention(heads, kv, d, d, dtype=TYPES[kind], device=DEV)
        s["cache"] = nys.PagedKV4(pages, page, kv, d, d, dtype=TYPES[kind], device=DEV, data=s["data"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["n"], heads), device=DEV)
    return s


def run(s):
    if own:
        if s["op"] == "norm":
            s["prepare"].rows(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if s["op"] == "append":
            s["prepare"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cache"], q_out=s["q_out"])
            return {"q": s["q_out"], "k": s["pool_k"], "v": s["pool_v"]}
        if s["op"] == "write4":
            s["cache"].write(s["k"], s["v"], s["slots"])
            s["cache"].read(s["every"], s["k_out"], s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        s["attention"].paged4(s["q"], s["cache"], s["lens"], s["table"], s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"norm": _norm, "append": _append, "write4": _write4, "attend4": _attend4}[s["op"]](s)


# ---------------------------------------------------------------- plain forms
def _norm_rotate(x, weight, positions, freqs, rot, inter):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight
    # Angles of far positions lose their digits in 32 bits.
    angle = positions.double()[:, None] * freqs
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    pair = x[..., :rot].unflatten(-1, (-1, 2)) if inter else x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
    a, b = pair[..., 0], pair[..., 1]
    turned = (a * cos - b * sin, a * sin + b * cos)
    turned = torch.stack(turned, dim=-1).flatten(-2) if inter else torch.cat(turned, dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _norm(s):
    to = lambda x, w: _norm_rotate(x, w, s["positions"], s["freqs"], s["rot"], s["inter"]).to(x.dtype)  # noqa: E731
    return {"q": to(s["q"], s["q_weight"]), "k": to(s["k"], s["k_weight"])}


def _append(s):
    turned = _norm(s)
    s["pool_k"].view(-1, *s["k"].shape[1:])[s["slots"]] = turned["k"]
    s["pool_v"].view(-1, *s["v"].shape[1:])[s["slots"]] = s["v"]
    return {"q": turned["q"], "k": s["pool_k"], "v": s["pool_v"]}


def _quantize(x):
    """Codes [..][d] and each group's step and middle [..][groups] of f32 rows [..][d]."""
    d, groups = x.shape[-1], -(-x.shape[-1] // 64)
    # A last group that is short is filled up with its own first number.
    first = x[..., 64 * (groups - 1):64 * (groups - 1) + 1]
    x = torch.cat([x, first.expand(*x.shape[:-1], 64 * groups - d)], dim=-1).unflatten(-1, (groups, 64))
    lo, hi = x.amin(dim=-1), x.amax(dim=-1)
    # Quotients next to a border decide on a code: divisions by tensors, which round correctly.
    mid = (lo + (hi - lo) * 8 / torch.full_like(lo, 15)).to(torch.bfloat16).float()
    step = torch.maximum((hi - mid) / torch.full_like(hi, 7), (mid - lo) * 0.125)
    step = ((step.view(torch.int32) + 0xffff) & -0x10000).view(torch.float32)
    step = torch.where(step < 2.0 ** -100, 0.0, step)
    codes = ((x - mid[..., None]) / torch.where(step > 0, step, 1.0)[..., None]).round()
    codes = torch.where(step[..., None] > 0, (codes + 8).clamp(0, 15), 8.0)
    return codes.flatten(-2)[..., :d], step, mid


def _dequantize(codes, step, mid):
    d = codes.shape[-1]
    spread = lambda x: x.repeat_interleave(64, dim=-1)[..., :d]  # noqa: E731
    return spread(mid) + spread(step) * (codes - 8)


def _rows4(data, kv, d, page):
    """All rows of a 4-bit cache: keys and values [slots][kv_heads][d] in f32."""
    groups = -(-d // 64)
    blocks = data.view(torch.int32).view(-1, kv, page // 16, 288 * groups)
    shifts = 4 * torch.arange(8, dtype=torch.int32, device=data.device)
    out = []
    for is_k, codes_at, scales_at in ((True, 0, 256 * groups), (False, 128 * groups, 272 * groups)):
        words = blocks[..., codes_at:codes_at + 128 * groups]
        if is_k:  # [page][kv][block][group][t][c][t8][h] -> [page][block][t8][t][kv][group][h][c]
            words = words.reshape(-1, kv, page // 16, groups, 8, 4, 2, 2).permute(0, 2, 6, 4, 1, 3, 7, 5)
        else:  # [page][kv][block][group][r][t2][t8][t1] -> [page][block][t8][t2][t1][kv][group][r]
            words = words.reshape(-1, kv, page // 16, groups, 8, 4, 2, 2).permute(0, 2, 6, 5, 7, 1, 3, 4)
        codes = ((words.reshape(-1, kv, 8 * groups, 1) >> shifts) & 15).flatten(-2)[..., :d].float()
        scale = blocks[..., scales_at:scales_at + 16 * groups].reshape(-1, kv, page // 16, groups, 4, 2, 2)
        scale = scale.permute(0, 2, 5, 4, 6, 1, 3).reshape(-1, kv, groups)
        out.append(_dequantize(codes, (scale & -0x10000).view(torch.float32), (scale << 16).view(torch.float32)))
    return out


def _write4(s):
    rows = _rows4(s["data"], s["kv_heads"], s["d"], s["page"])
    for x, new in zip(rows, (s["k"], s["v"])):
        x[s["slots"]] = _dequantize(*_quantize(new.float()))
    return {"k": rows[0].to(s["k"].dtype), "v": rows[1].to(s["k"].dtype)}


def _attend4(s):
    q, kv, page = s["q"], s["kv_heads"], s["page"]
    n, heads, d = q.shape
    table = s["table"].long().clamp(min=0)
    ks, vs = _rows4(s["data"], kv, d, page)
    ks = ks.view(-1, page, kv, d)[table].view(n, -1, kv, d)
    vs = vs.view(-1, page, kv, d)[table].view(n, -1, kv, d)
    scores = torch.einsum("bkgd,btkd->bkgt", q.float().view(n, kv, heads // kv, d), ks) * (1.0 / math.sqrt(d))
    beyond = torch.arange(ks.shape[1], device=DEV) >= s["lens"][:, None]
    scores.masked_fill_(beyond[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = (scores - top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = torch.einsum("bkgt,btkd->bkgd", p, vs) / total
    return {"out": out.reshape(n, heads, d).to(q.dtype), "lse": (top + total.log()).reshape(n, heads)}


# ---------------------------------------------------------------- floors
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}[case["type"]]
    kv, d = case["kv_heads"], case["d"]
    held = 2 * kv * (d / 2 + 4 * -(-d // 64))  # bytes of a token in the 4-bit cache
    if case["op"] == "attend4":
        keys = sum(_lengths(case))
        return {"bytes": 2 * case["n"] * case["heads"] * d * size + keys * held, "flops": 4 * case["heads"] * d * keys}
    tokens = case["tokens"]
    if case["op"] == "write4":
        # Rows in, their bytes written; all bytes read (about the new rows'), all values out.
        row = 2 * kv * d * size
        return {"bytes": tokens * (2 * row + 2 * held + 8), "flops": 0}
    rows = case["heads"] + kv + (kv if case["op"] == "append" else 0)
    return {"bytes": tokens * (2 * rows * d * size + 4 + (8 if case["op"] == "append" else 0)), "flops": 0}


# ---------------------------------------------------------------- 64-bit forms
def _turn64(x, weight, positions, freqs, inter):
    """Norm and rotation of [rows][heads][d] in float64, pair by pair as complex numbers."""
    x = x.double()
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
    half = len(freqs)
    angle = (positions.double()[:, None] * freqs)[:, None, :]
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _held64(x):
    """The values that a 4-bit cache holds for rows [..][d], group by group in float64."""
    y = x.double().clone()
    for at in range(0, x.shape[-1], 64):
        part = y[..., at:at + 64]
        lo, hi = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        mid = (lo + (hi - lo) * 8 / 15).to(torch.bfloat16).double()
        need = torch.maximum((hi - mid) / 7, (mid - lo) / 8)
        step = need.to(torch.bfloat16)
        up = torch.nextafter(step, torch.full_like(step, math.inf))
        step = torch.where(step.double() < need, up, step).double()
        code = torch.round((part - mid) / torch.where(step > 0, step, 1.0)).clamp(-8, 7)
        y[..., at:at + 64] = mid + step * code
    return y


def _row64(data, slots, page, kv, d, values):
    """Rows [slots][kv_heads][d] of a 4-bit cache in float64, each code looked up at its own place."""
    groups = -(-d // 64)
    blocks = data.view(torch.int32).view(-1, 288 * groups)
    page_no, at = slots // page, slots % page
    block = (page_no[:, None] * kv + torch.arange(kv, device=data.device)) * (page // 16) + (at // 16)[:, None]
    t = (at % 16)[:, None]
    x = torch.arange(d, device=data.device)
    g, e = x // 64, x % 64
    place = (t % 8 // 2) * 4 + t // 8 * 2 + t % 2
    if values:
        word = 128 * groups + g * 128 + e // 8 * 16 + place
    else:
        word = g * 128 + t % 8 * 16 + e % 32 // 8 * 4 + t // 8 * 2 + e // 32
    codes = (blocks[block[:, :, None], word[:, None, :]] >> (4 * (e % 8))) & 15
    scale = blocks[block[:, :, None], ((272 if values else 256) * groups + g * 16 + place)[:, None, :]]
    step, mid = ((scale >> 16) << 16).view(torch.float32).double(), (scale << 16).view(torch.float32).double()
    return mid + step * (codes - 8)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "append"):
        q = _turn64(s["q"], s["q_weight"], s["positions"], s["freqs"], case["inter"])
        k = _turn64(s["k"], s["k_weight"], s["positions"], s["freqs"], case["inter"])
        if case["op"] == "norm":
            return {"q": q, "k": k}
        page = case["page"]
        pools = [s["pool_k"].double(), s["pool_v"].double()]
        for pool, x in zip(pools, (k, s["v"].double())):
            pool[s["slots"] // page, s["slots"] % page] = x
        return {"q": q, "k": pools[0], "v": pools[1]}
    kv, d, page = case["kv_heads"], case["d"], case["page"]
    if case["op"] == "write4":
        rows = [_row64(s["data"], s["every"], page, kv, d, values) for values in (False, True)]
        for x, new in zip(rows, (s["k"], s["v"])):
            x[s["slots"]] = _held64(new)
        return {"k": rows[0], "v": rows[1]}
    heads, n = case["heads"], case["n"]
    q = s["q"].double().view(n, kv, heads // kv, d)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device=DEV)
    for i, count in enumerate(s["lens"].tolist()):
        j = torch.arange(count, device=DEV)
        slots = s["table"][i].long()[j // page] * page + j % page
        k, v = (_row64(s["data"], slots, page, kv, d, values) for values in (False, True))
        scores = (q[i].unsqueeze(2) * k.transpose(0, 1).unsqueeze(1)).sum(-1) / math.sqrt(d)
        lse[i] = torch.logsumexp(scores, -1)
        out[i] = (torch.exp(scores - lse[i].unsqueeze(-1)).unsqueeze(-1) * v.transpose(0, 1).unsqueeze(1)).sum(2)
    return {"out": out.view(n, heads, d), "lse": lse.view(n, heads)}
