"""The tiled attention kernels' bounded waits, made to run out on purpose.

nys_debug_stall_attn_once makes the next launch's first CTA issue no copies, or no
products: its warps wait for what never comes, give up after 2 s, set the status
word, drain what is in flight, free their tensor memory and return; nothing faults
and the CUDA context stays usable.  Other CTAs' rows come out as ever, and the next
call is right everywhere.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

COPIES, PRODUCTS = 1, 2


def _mods():
    import torch
    import attn_reference as ref
    from streaming_nystr_landmark_gb300 import nys
    return torch, ref, nys


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("role", [COPIES, PRODUCTS])
def test_stalled_prompt_gives_up_and_says_so(cuda_device, dtype, role):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    heads, kv, d, n, length = 4, 2, 64, 200, 90
    g = torch.Generator(device=cuda_device).manual_seed(0)
    q, k, v = (torch.randn((n * length, h, d), generator=g, device=cuda_device).to(dt)
               for h in (heads, kv, kv))
    off = (torch.arange(n + 1, device=cuda_device) * length).int()
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    want, out = torch.empty_like(q), torch.full_like(q, 7.0)
    att.prompt(q, k, v, off, want)
    assert att.status() == 0
    nys.nys_debug_stall_attn_once(role)
    att.prompt(q, k, v, off, out)
    torch.cuda.synchronize()          # the stalled CTA returned: the context is alive
    assert att.status() == nys.NYS_ATTN_GAVE_UP
    # Whole rows of a KV head were written as ever or left alone: at most the units
    # that the first CTA had taken (three in a ring, one more begun) of 64 rows of
    # two heads or more.
    same = (out == want).view(n * length, kv, -1).all(-1)
    left = (out == 7.0).view(n * length, kv, -1).all(-1)
    assert bool((same | left).all())
    assert 0 < int(left.sum()) <= 4 * 128
    att.clear_status()
    out.fill_(7.0)
    att.prompt(q, k, v, off, out)
    assert torch.equal(out, want) and att.status() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("role", [COPIES, PRODUCTS])
def test_stalled_prefix_gives_up_and_says_so(cuda_device, dtype, role):
    torch, ref, nys = _mods()
    dt = getattr(torch, dtype)
    n, heads, kv, d, page, prefix = 300, 4, 2, 64, 16, 512
    g = torch.Generator(device=cuda_device).manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device).to(dt)
    q = rn(n, heads, d)
    cache = nys.PagedKV(prefix // page, page, kv, d, d, dtype=dt, device=cuda_device,
                        k=rn(prefix // page, page, kv, d), v=rn(prefix // page, page, kv, d))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    att = nys.ExactAttention(heads, kv, d, d, dtype=dt, device=cuda_device)
    args = (q, cache, i32([0] * n), i32([[0]] * n))
    more = dict(prefix_pages=i32(list(range(prefix // page))), prefix_len=prefix)
    want, out = torch.empty_like(q), torch.empty_like(q)
    att.shared(*args, want, **more)
    assert att.status() == 0
    nys.nys_debug_stall_attn_once(role)
    att.shared(*args, out, **more)
    torch.cuda.synchronize()
    assert att.status() == nys.NYS_ATTN_GAVE_UP
    att.clear_status()
    att.shared(*args, out, **more)
    assert torch.equal(out, want) and att.status() == 0
