"""The exact side of one attention layer in a serving loop.

A landmark state (nys.NystromStates) replaces a request's KV cache once its
prompt is sealed; until then, and for layers and requests that stay exact, a
server needs what this module puts together from the exact operators of
nys.py: a pool of KV pages with a prefix that all requests share, the admission
of prompts of any lengths, and one-token decode.

    layer = ExactLayer(heads=16, kv_heads=8, d=128, dv=128, requests=64, ...)
    layer.set_prefix(k, v)                    # a system prompt, once
    out = layer.admit(q, k, v, lengths)       # packed prompts of all requests
    out = layer.decode(q, k, v)               # one token for each of them
    seal_prompts(states, q, k, v, lengths)    # landmark states of the same prompts

Everything is enqueued on the current torch stream; the host only counts
pages, so nothing waits for the GPU.  What only the GPU can see (a wait that ran
out, a page outside the pool) is in layer.status().
"""
from __future__ import annotations

from . import nys


def merge(out_a, lse_a, out_b, lse_b, out):
    """Attention over two disjoint sets of keys from the results over each and
    their log-sums: sum_x e^{lse_x} out_x / sum_x e^{lse_x}, in f32; rows that
    saw neither set stay 0.  Results of 16-bit types come rounded to their type,
    so the sum of two is off by up to half a step more than one pass over all keys
    would be: that pass would have to read the prefix from its pages for every
    prompt row, which the operators do for single tokens."""
    import torch
    top = torch.maximum(lse_a, lse_b)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    wa, wb = torch.exp(lse_a - top), torch.exp(lse_b - top)
    total = wa + wb
    total = torch.where(total == 0, torch.ones_like(total), total)
    a = (wa / total).unsqueeze(-1) * out_a.float()
    out.copy_(a.addcmul_((wb / total).unsqueeze(-1), out_b.float()))
    return out


class ExactLayer:
    """One layer's exact attention for `requests` requests of up to max_len
    tokens each (besides the shared prefix), in pages of `page` tokens.  It serves
    one batch: requests are admitted together, each gets a token in every decode,
    and pages are given back with the object."""

    def __init__(self, heads, kv_heads, d, dv, requests, n_pages, page, max_len, dtype=None,
                 scale=None, device="cuda"):
        import torch
        self.torch = torch
        self.device = nys._cuda_device(device)
        self.attention = nys.ExactAttention(heads, kv_heads, d, dv, dtype=dtype, scale=scale,
                                            device=self.device)
        self.cache = nys.PagedKV(n_pages, page, kv_heads, d, dv, dtype=dtype, device=self.device)
        self.requests, self.page = requests, page
        self.width = -(-max_len // page)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.table = torch.full((requests, self.width), -1, **i32)
        self.free = torch.arange(n_pages, **i32)
        self.used = 0                       # pages taken from the front of `free`
        self.lengths = [0] * requests       # tokens of each request, as the host counts them
        self.lens = torch.zeros(requests, **i32)
        self.prefix_len = 0
        self.prefix_pages = None
        self._plans = {}

    def status(self):
        """The status bits (NYS_ATTN_*, NYS_PLAN_*) of all calls since the last clear;
        synchronises.  Anything but 0 means that results are not to be used; a
        server looks at it where it reads results anyway."""
        return self.attention.status()

    def clear_status(self):
        self.attention.clear_status()

    def _check(self, q, k, v):
        """Refuses tensors that a call below would refuse, before anything is taken
        or counted."""
        att, index = self.attention, self.device.index
        if q is not None:
            nys._rows(q, att.dtype, att.heads, att.d, "q", index)
        nys._rows(k, att.dtype, att.kv_heads, att.d, "k", index)
        nys._rows(v, att.dtype, att.kv_heads, att.dv, "v", index)
        if v.shape[0] != k.shape[0]:
            raise ValueError(f"v: {v.shape[0]} rows, k has {k.shape[0]}")

    def _plan(self, fresh):
        """Pages and slots for fresh[i] more tokens of request i."""
        torch, total = self.torch, sum(fresh)
        if len(fresh) != self.requests or min(fresh) < 0:
            raise ValueError(f"need {self.requests} lengths, none negative")
        pages = lambda n: -(-n // self.page)
        need = sum(pages(a + b) - pages(a) for a, b in zip(self.lengths, fresh))
        if self.used + need > self.free.shape[0]:
            raise ValueError(f"{need} more pages wanted, {self.free.shape[0] - self.used} left")
        if max(a + b for a, b in zip(self.lengths, fresh)) > self.width * self.page:
            raise ValueError("a request would outgrow max_len")
        if total not in self._plans:
            plan = nys.PagePlan(self.requests, self.width, total, self.page, device=self.device)
            plan.share_status(self.attention)
            self._plans = {total: plan}
        plan = self._plans[total]
        # From pinned memory: a copy that the host does not wait for.
        grow = torch.tensor(fresh, dtype=torch.int32, pin_memory=True).to(self.device,
                                                                         non_blocking=True)
        plan.update(self.lens, grow, self.free[self.used:], self.table)
        self.used += need
        self.lengths = [a + b for a, b in zip(self.lengths, fresh)]
        self.lens.copy_(plan.lens)
        return plan

    def set_prefix(self, k, v):
        """Keys and values [rows][kv_heads][d|dv] that every request sees first;
        before any request is admitted."""
        if self.used:
            raise ValueError("the prefix comes before the first request")
        self._check(None, k, v)
        torch, n = self.torch, k.shape[0]
        need = -(-n // self.page)
        if need > self.free.shape[0]:
            raise ValueError(f"{need} pages wanted, {self.free.shape[0]} there")
        pages = self.free[:need].clone()
        at = torch.arange(n, device=self.device)
        self.cache.write(k, v, pages.long()[at // self.page] * self.page + at % self.page)
        self.used, self.prefix_pages, self.prefix_len = need, pages, n

    def admit(self, q, k, v, lengths):
        """The requests' prompts, packed back to back (q [sum][heads][d], k and v
        [sum][kv_heads][d|dv]): into their pages, and attended causally after the
        prefix.  Returns [sum][heads][dv]."""
        torch, att = self.torch, self.attention
        if any(self.lengths):
            raise ValueError("admit() takes requests from their first token")
        if not q.shape[0] == k.shape[0] == v.shape[0] == sum(lengths):
            raise ValueError("q, k and v must have as many rows as the lengths' sum")
        self._check(q, k, v)
        # Memory first: an allocation that fails leaves the requests as they were.
        rows = q.shape[0]
        out = torch.empty((rows, att.heads, att.dv), dtype=att.dtype, device=self.device)
        att._workspace(self.requests, rows, rows)
        if self.prefix_len > 0:
            lse, over = torch.empty((2, rows, att.heads), device=self.device).unbind(0)
            first = torch.empty_like(out)
            none = torch.zeros(rows, dtype=torch.int32, device=self.device)
            att._workspace(rows, rows, self.prefix_len)
        plan = self._plan(list(lengths))
        self.cache.write(k, v, plan.slots)
        if self.prefix_len == 0:
            return att.prompt(q, k, v, plan.q_off, out)
        # Over the prompt's own keys and, as rows without own keys, over the prefix.
        att.prompt(q, k, v, plan.q_off, out, lse=lse)
        att.shared(q, self.cache, none, none.view(rows, 1), first,
                   prefix_pages=self.prefix_pages, prefix_len=self.prefix_len, lse=over)
        return merge(out, lse, first, over, out)

    def decode(self, q, k, v):
        """One new token for every request: q [requests][heads][d], k and v
        [requests][kv_heads][d|dv].  Returns [requests][heads][dv]."""
        att = self.attention
        if not q.shape[0] == k.shape[0] == v.shape[0] == self.requests:
            raise ValueError("q, k and v must have one row a request")
        self._check(q, k, v)
        out = self.torch.empty((self.requests, att.heads, att.dv), dtype=att.dtype,
                               device=self.device)
        att._workspace(self.requests, self.requests, self.prefix_len)
        plan = self._plan([1] * self.requests)
        self.cache.write(k, v, plan.slots)
        return att.shared(q, self.cache, self.lens, self.table, out,
                          prefix_pages=self.prefix_pages, prefix_len=self.prefix_len)


def seal_prompts(states, q, k, v, lengths, g0=0):
    """Seals landmark states on packed prompts (the tensors of
    ExactLayer.admit; 16-bit ones as the f32 values they hold, which the states
    keep): request i's KV head j becomes group g0 + i * kv_heads + j of `states`."""
    import torch
    rows, heads, d = q.shape
    if not rows == k.shape[0] == v.shape[0] == sum(lengths):
        raise ValueError("q, k and v must have as many rows as the lengths' sum")
    kv, group = k.shape[1], heads // k.shape[1]
    qs, ks, vs = [], [], []
    at = 0
    for t in lengths:
        cut = slice(at, at + t)
        qs.append(q[cut].view(t, kv, group, d).permute(1, 2, 0, 3).reshape(-1, d))
        ks.append(k[cut].transpose(0, 1).reshape(-1, d))
        vs.append(v[cut].transpose(0, 1).reshape(-1, v.shape[2]))
        at += t
    states.seal_ragged([t for t in lengths for _ in range(kv)], torch.cat(qs).float(),
                       torch.cat(ks).float(), torch.cat(vs).float(), g0=g0)
