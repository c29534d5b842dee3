"""The exact-attention operators that stand next to the landmark states, as
measured workloads: their inputs, their plain form and their 64-bit form.

  prompt   causal attention of packed prompts with grouped heads
  shared   one token of attention for a batch that shares a prefix; the
           prefix and every request's own keys sit in pages of one pool
  plan     block tables, slots and positions from request lengths
  write    new keys and values into the pages of their slots

``listed()`` gives the fixed cases, ``draw()`` more of the same ranges.  With
``own`` false ``run`` computes an operator in elementary torch operations,
with ``own`` true it makes the calls of streaming_nystr_landmark_gb300.nys.
Geometries are those of workloads.py: 16 query heads over 8 KV heads with
head dim 128 (``layer``, ``batch64``), 32 over 4 (``long``), 1 over 1 with
head dim 64 (``single``).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # One short prompt of the smallest geometry: a launch's latency.
        {"name": "prompt single f32", "op": "prompt", "type": "f32", "heads": 1, "kv_heads": 1, "d": 64,
         "n": 1, "lo": 64, "hi": 64, "cached": 0},
        # The prompts of batch64's layers, in the framework's own type: many short sequences.
        {"name": "prompt batch f32", "op": "prompt", "type": "f32", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 64, "lo": 256, "hi": 256, "cached": 0},
        # Requests of every length in one packed batch, as a server admits them.
        {"name": "prompt ragged bf16", "op": "prompt", "type": "bf16", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 33, "lo": 1, "hi": 2047, "cached": 0},
        # The last part of a long prompt that is taken in parts: its keys are already there.
        {"name": "prompt continued f32", "op": "prompt", "type": "f32", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 2, "lo": 1021, "hi": 1500, "cached": 5003},
        # One long prompt at the long-context geometry.
        {"name": "prompt long bf16", "op": "prompt", "type": "bf16", "heads": 32, "kv_heads": 4, "d": 128,
         "n": 1, "lo": 16384, "hi": 16384, "cached": 0},
        # A handful of requests under a short system prompt: latency.
        {"name": "shared few bf16", "op": "shared", "type": "bf16", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 4, "lo": 3, "hi": 45, "prefix": 301, "page": 16},
        # 64 chats under one system prompt, in the framework's own type.
        {"name": "shared chats f32", "op": "shared", "type": "f32", "heads": 16, "kv_heads": 8, "d": 128,
         "n": 64, "lo": 97, "hi": 1025, "prefix": 2000, "page": 16},
        # Many questions about one long document.
        {"name": "shared document bf16", "op": "shared", "type": "bf16", "heads": 32, "kv_heads": 4, "d": 128,
         "n": 256, "lo": 1, "hi": 517, "prefix": 32768, "page": 64},
        # A decode step's bookkeeping: one new token for each of 64 requests.
        {"name": "plan decode", "op": "plan", "n": 64, "lo": 1, "hi": 1, "cached": 4000, "page": 16},
        # Admission of many prompts at once.
        {"name": "plan admission", "op": "plan", "n": 1000, "lo": 1, "hi": 1024, "cached": 0, "page": 64},
        # A decode step's new rows.
        {"name": "write decode f32", "op": "write", "type": "f32", "kv_heads": 8, "d": 128, "tokens": 64, "page": 16},
        # A batch of prompts' rows.
        {"name": "write prompts bf16", "op": "write", "type": "bf16", "kv_heads": 8, "d": 128, "tokens": 16384,
         "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "shared", "shared", "shared", "plan", "write"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "plan":
        lo = _log(rng, 1, 300)
        return {"op": op, "n": _log(rng, 1, 1500), "lo": lo, "hi": _log(rng, lo, 600),
                "cached": rng.choice([0, _log(rng, 1, 8000)]), "page": page}
    kind = rng.choice(list(TYPES))
    heads, kv_heads = rng.choice([(16, 8), (32, 4), (1, 1), (8, 8), (12, 4), (14, 2), (24, 8)])
    d = rng.choice([64, 128, 128, 96, 80])
    if op == "write":
        return {"op": op, "type": kind, "kv_heads": kv_heads, "d": d, "tokens": _log(rng, 1, 20000), "page": page}
    n = _log(rng, 1, 64) if op == "prompt" else _log(rng, 1, 200)
    if op == "prompt":
        hi = _log(rng, 1, min(4096, 16384 // n))
        cached = rng.choice([0, 0, _log(rng, 1, 2048)])
        return {"op": op, "type": kind, "heads": heads, "kv_heads": kv_heads, "d": d, "n": n,
                "lo": _log(rng, 1, hi), "hi": hi, "cached": cached}
    hi = _log(rng, 1, min(4096, 65536 // n))
    return {"op": op, "type": kind, "heads": heads, "kv_heads": kv_heads, "d": d, "n": n, "lo": _log(rng, 1, hi),
            "hi": hi, "prefix": rng.choice([0, _log(rng, 1, 16384), _log(rng, 1, 16384)]), "page": page}


def _lengths(case):
    """The batch's lengths, spread geometrically from hi down to lo."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    return [int(round(hi * (lo / hi) ** (i / max(1, n - 1)))) for i in range(n)]


def _shuffled(values, seed):
    order = np.random.RandomState(seed % (1 << 31)).permutation(len(values))
    return [values[i] for i in order]


def _offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)


def _randn(gen, shape, kind):
    return torch.randn(shape, generator=gen, device=DEV).to(TYPES[kind])


def _keys(gen, rows, kv_heads, d, kind):
    """Keys with a mean direction for each head, as workloads.py draws them."""
    u = torch.randn((1, kv_heads, d), generator=gen, device=DEV)
    k = torch.randn((rows, kv_heads, d), generator=gen, device=DEV)
    return (k + 2.0 * u / u.norm(dim=-1, keepdim=True)).to(TYPES[kind])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    make = {"prompt": _prepare_prompt, "shared": _prepare_shared, "plan": _prepare_plan, "write": _prepare_write}
    state = make[case["op"]](case, gen, int(seed))
    state["op"] = case["op"]
    return state


def _prepare_prompt(case, gen, seed):
    heads, kv_heads, d, kind = case["heads"], case["kv_heads"], case["d"], case["type"]
    new = _shuffled(_lengths(case), seed)
    have = [x + case["cached"] for x in new]
    s = {"q": _randn(gen, (sum(new), heads, d), kind), "k": _keys(gen, sum(have), kv_heads, d, kind),
         "v": _randn(gen, (sum(have), kv_heads, d), kind), "q_off": _offsets(new), "k_off": _offsets(have),
         "most": max(new), "most_keys": max(have)}
    if own:
        from streaming_nystr_landmark_gb300 import nys
        s["attention"] = nys.ExactAttention(heads, kv_heads, d, d, dtype=TYPES[kind], device=DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device=DEV)
    return s


def _prepare_shared(case, gen, seed):
    heads, kv_heads, d, kind, page = case["heads"], case["kv_heads"], case["d"], case["type"], case["page"]
    lengths = _shuffled(_lengths(case), seed)
    need = [-(-x // page) for x in lengths]
    first = -(-case["prefix"] // page)
    width = max(max(need), 1)
    pages = first + sum(need) + 3
    order = np.random.RandomState((seed + 1) % (1 << 31)).permutation(pages)
    table = np.full((case["n"], width), -1, dtype=np.int32)
    at = first
    for i, x in enumerate(need):
        table[i, :x] = order[at:at + x]
        at += x
    s = {"q": _randn(gen, (case["n"], heads, d), kind),
         "k": _keys(gen, pages * page, kv_heads, d, kind).view(pages, page, kv_heads, d),
         "v": _randn(gen, (pages, page, kv_heads, d), kind),
         "lens": torch.tensor(lengths, dtype=torch.int32, device=DEV),
         "table": torch.tensor(table, device=DEV),
         "prefix_pages": torch.tensor(order[:first].astype(np.int32), device=DEV), "prefix": case["prefix"]}
    if own:
        from streaming_nystr_landmark_gb300 import nys
        s["attention"] = nys.ExactAttention(heads, kv_heads, d, d, dtype=TYPES[kind], device=DEV)
        s["cache"] = nys.PagedKV(pages, page, kv_heads, d, d, dtype=TYPES[kind], device=DEV, k=s["k"], v=s["v"])
        s["out"] = torch.empty_like(s["q"])
    return s


def _prepare_plan(case, gen, seed):
    page, n = case["page"], case["n"]
    fresh = _shuffled(_lengths(case), seed)
    rs = np.random.RandomState((seed + 1) % (1 << 31))
    # Requests of any age around the mean length, so that pages end anywhere.
    cached = rs.permutation(np.linspace(0, 2 * case["cached"], n).round().astype(np.int64))
    old = -(-cached // page)
    new = -(-(cached + np.array(fresh)) // page)
    width = int(-(-(2 * case["cached"] + max(fresh)) // page))
    pages = int(new.sum()) + 7
    order = rs.permutation(pages).astype(np.int32)
    table = np.full((n, width), -1, dtype=np.int32)
    held = np.arange(width)[None, :] < old[:, None]
    table[held] = order[:int(old.sum())]
    free = order[int(old.sum()):]
    total = int(sum(fresh))
    t = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)  # noqa: E731
    s = {"cached": t(cached), "fresh": t(fresh), "free": t(free), "table": t(table), "page": page, "total": total}
    if own:
        from streaming_nystr_landmark_gb300 import nys
        s["plan"] = nys.PagePlan(n, width, total, page, device=DEV)
    return s


def _prepare_write(case, gen, seed):
    kv_heads, d, kind, page, tokens = case["kv_heads"], case["d"], case["type"], case["page"], case["tokens"]
    pages = -(-tokens // page) + 3
    slots = torch.randperm(pages * page, generator=gen, device=DEV)[:tokens]
    s = {"k": _randn(gen, (tokens, kv_heads, d), kind), "v": _randn(gen, (tokens, kv_heads, d), kind), "slots": slots,
         "pool_k": _randn(gen, (pages, page, kv_heads, d), kind),
         "pool_v": _randn(gen, (pages, page, kv_heads, d), kind)}
    if own:
        from streaming_nystr_landmark_gb300 import nys
        s["cache"] = nys.PagedKV(pages, page, kv_heads, d, d, dtype=TYPES[kind], device=DEV, k=s["pool_k"],
                                 v=s["pool_v"])
    return s


def run(s):
    if own:
        if s["op"] == "prompt":
            s["attention"].prompt(s["q"], s["k"], s["v"], s["q_off"], s["out"], k_off=s["k_off"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if s["op"] == "shared":
            return s["attention"].shared(s["q"], s["cache"], s["lens"], s["table"], s["out"],
                                         prefix_pages=s["prefix_pages"], prefix_len=s["prefix"])
        if s["op"] == "plan":
            p = s["plan"]
            p.update(s["cached"], s["fresh"], s["free"], s["table"])
            return {"table": s["table"], "q_off": p.q_off, "lens": p.lens, "slots": p.slots, "positions": p.positions,
                    "taken": p.taken}
        s["cache"].write(s["k"], s["v"], s["slots"])
        return {"k": s["pool_k"], "v": s["pool_v"]}
    return {"prompt": _prompt, "shared": _shared, "plan": _plan, "write": _write}[s["op"]](s)


# ---------------------------------------------------------------- plain forms
def _softmax_sums(scores):
    """exp(scores - max), its sum and the log of the whole sum; rows of -inf give zeros."""
    top = scores.amax(dim=-1, keepdim=True)
    p = (scores - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    return p, total, (top + total.log()).squeeze(-1)


def _prompt(s):
    q, k, v, q_off, k_off = s["q"], s["k"], s["v"], s["q_off"].long(), s["k_off"].long()
    (rows, heads, d), kv_heads = q.shape, k.shape[1]
    n, group = len(q_off) - 1, heads // kv_heads
    nq, nk = q_off[1:] - q_off[:-1], k_off[1:] - k_off[:-1]
    # Padded to one rectangle a sequence; rows past a sequence's end repeat its edge and are masked.
    iq, ik = torch.arange(s["most"], device=DEV), torch.arange(s["most_keys"], device=DEV)
    qp = q[(q_off[:-1, None] + iq).clamp(max=rows - 1)].float()
    at = (k_off[:-1, None] + ik).clamp(max=len(k) - 1)
    kp, vp = k[at].float(), v[at].float()
    qp = qp.view(n, -1, kv_heads, group, d).permute(0, 2, 3, 1, 4).reshape(n, kv_heads, -1, d)
    scores = torch.matmul(qp, kp.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    scores = scores.view(n, kv_heads, group, s["most"], s["most_keys"])
    seen = (ik <= iq[:, None] + (nk - nq)[:, None, None]) & (ik < nk[:, None, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    p, total, lse = _softmax_sums(scores)
    out = torch.matmul(p.view(n, kv_heads, -1, s["most_keys"]), vp.transpose(1, 2))
    out = out.view(n, kv_heads, group, -1, d) / torch.where(total == 0, 1.0, total)
    token = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(q_off[1:], token, right=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, -1, heads, d)[seq, token - q_off[seq]]
    lse = lse.permute(0, 3, 1, 2).reshape(n, -1, heads)[seq, token - q_off[seq]]
    return {"out": out.to(q.dtype), "lse": lse}


def _shared(s):
    q, k, v = s["q"], s["k"], s["v"]
    (n, heads, d), kv_heads, page = q.shape, k.shape[2], k.shape[1]
    group, scale = heads // kv_heads, 1.0 / math.sqrt(d)
    qf = q.float().view(n, kv_heads, group, d)
    # The prefix once for all requests.
    at = s["prefix_pages"].long()
    kp = k[at].float().reshape(-1, kv_heads, d)[:s["prefix"]]
    vp = v[at].float().reshape(-1, kv_heads, d)[:s["prefix"]]
    first = torch.einsum("bkgd,tkd->bkgt", qf, kp) * scale
    # Every request's own pages.
    table = s["table"].long().clamp(min=0)
    ko = k[table].float().reshape(n, -1, kv_heads, d)
    vo = v[table].float().reshape(n, -1, kv_heads, d)
    then = torch.einsum("bkgd,btkd->bkgt", qf, ko) * scale
    beyond = torch.arange(ko.shape[1], device=DEV) >= s["lens"][:, None]
    then.masked_fill_(beyond[:, None, None], -math.inf)
    p, total, _ = _softmax_sums(torch.cat([first, then], dim=-1))
    out = torch.einsum("bkgt,tkd->bkgd", p[..., :len(kp)], vp) + torch.einsum("bkgt,btkd->bkgd", p[..., len(kp):], vo)
    return (out / torch.where(total == 0, 1.0, total)).reshape(n, heads, d).to(q.dtype)


def _plan(s):
    cached, fresh, free, page = s["cached"].long(), s["fresh"].long(), s["free"], s["page"]
    old, new = (cached + page - 1) // page, (cached + fresh + page - 1) // page
    ends = (new - old).cumsum(0)
    column = torch.arange(s["table"].shape[1], device=DEV)
    rank = (ends - new)[:, None] + column
    given = torch.where(rank < len(free), free[rank.clamp(0, len(free) - 1)], -1)
    s["table"].copy_(torch.where((column >= old[:, None]) & (column < new[:, None]), given, s["table"]))
    off = torch.cat([fresh.new_zeros(1), fresh.cumsum(0)])
    request = torch.repeat_interleave(torch.arange(len(fresh), device=DEV), fresh, output_size=s["total"])
    position = cached[request] + torch.arange(s["total"], device=DEV) - off[request]
    at = s["table"][request, position // page].long()
    slots = torch.where(at < 0, -1, at * page + position % page)
    return {"table": s["table"], "q_off": off.int(), "lens": (cached + fresh).int(), "slots": slots,
            "positions": position.int(), "taken": ends[-1:].clamp(max=len(free)).int()}


def _write(s):
    s["pool_k"].view(-1, *s["k"].shape[1:])[s["slots"]] = s["k"]
    s["pool_v"].view(-1, *s["v"].shape[1:])[s["slots"]] = s["v"]
    return {"k": s["pool_k"], "v": s["pool_v"]}


# ---------------------------------------------------------------- floors
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}[case.get("type", "f32")]
    if case["op"] == "write":
        row = case["tokens"] * case["kv_heads"] * case["d"] * size
        return {"bytes": 4 * row + 8 * case["tokens"], "flops": 0}
    lengths = _lengths(case)
    if case["op"] == "plan":
        page = case["page"]
        # Lengths in, offsets and lengths out; a page's number read and written; a slot and a position a token.
        return {"bytes": 16 * case["n"] + 8 * sum(lengths) / page + 12 * sum(lengths), "flops": 0}
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "prompt":
        new, have = sum(lengths), sum(lengths) + case["n"] * case["cached"]
        pairs = sum(x * (x + 1) // 2 + x * case["cached"] for x in lengths)
        return {"bytes": (2 * new * heads + 2 * have * kv_heads) * d * size + 4 * new * heads,
                "flops": 4 * heads * d * pairs}
    keys = case["prefix"] + sum(lengths)
    return {"bytes": (2 * case["n"] * heads + 2 * keys * kv_heads) * d * size,
            "flops": 4 * heads * d * (case["n"] * case["prefix"] + sum(lengths))}


# ---------------------------------------------------------------- 64-bit forms
def _attend64(q, k, v, causal_from=None):
    """softmax(q k' / sqrt d) v and its log-sum in float64: q [r][d], k [t][d];
    row i sees keys 0 .. i + causal_from, or all where that is None."""
    if not len(k):
        return q.new_zeros((len(q), v.shape[1]), dtype=torch.float64), q.new_full((len(q),), -math.inf, dtype=torch.float64)
    s = (q.double() @ k.double().T) / math.sqrt(q.shape[1])
    if causal_from is not None:
        i, j = torch.arange(len(q), device=s.device), torch.arange(len(k), device=s.device)
        s[j[None, :] > i[:, None] + causal_from] = -math.inf
    lse = torch.logsumexp(s, dim=1)
    w = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return w @ v.double(), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "write":
        k, v = s["pool_k"].double(), s["pool_v"].double()
        page = case["page"]
        k[s["slots"] // page, s["slots"] % page] = s["k"].double()
        v[s["slots"] // page, s["slots"] % page] = s["v"].double()
        return {"k": k, "v": v}
    q, k, v = s["q"], s["k"], s["v"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    if case["op"] == "prompt":
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
        a, b = s["q_off"].tolist(), s["k_off"].tolist()
        for i in range(case["n"]):
            kk, vv = k[b[i]:b[i + 1]], v[b[i]:b[i + 1]]
            for h in range(case["heads"]):
                out[a[i]:a[i + 1], h], lse[a[i]:a[i + 1], h] = _attend64(
                    q[a[i]:a[i + 1], h], kk[:, h // group], vv[:, h // group], case["cached"])
        return {"out": out, "lse": lse}
    page = case["page"]
    k, v = k.reshape(-1, case["kv_heads"], case["d"]), v.reshape(-1, case["kv_heads"], case["d"])
    slots = lambda pages, count: (pages.long()[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:count]  # noqa: E731
    first = slots(s["prefix_pages"], case["prefix"])
    for h in range(case["kv_heads"]):
        rows = slice(h * group, (h + 1) * group)
        o1, l1 = _attend64(q[:, rows].reshape(-1, case["d"]), k[first, h], v[first, h])
        o1, l1 = o1.view(case["n"], group, -1), l1.view(case["n"], group)
        for i, count in enumerate(s["lens"].tolist()):
            mine = slots(s["table"][i], count)
            o2, l2 = _attend64(q[i, rows], k[mine, h], v[mine, h])
            lse = torch.logaddexp(l1[i], l2)
            out[i, rows] = o1[i] * (l1[i] - lse).exp()[:, None] + o2 * (l2 - lse).exp()[:, None]
    return out
