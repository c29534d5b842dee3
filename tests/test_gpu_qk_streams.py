"""QKPrepare's own copies of weights and turns, on streams other than the one it was made on."""
import pytest

pytestmark = pytest.mark.gpu

WAIT = 100_000_000   # cycles: 50 ms and more


def _set(dev):
    import torch
    from streaming_nystr_landmark_gb300 import nys
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((9, 2, 64), generator=g, device=dev)
    pos = torch.arange(9, dtype=torch.int32, device=dev)
    rotation = nys.Rotation(64, device=dev)
    make = lambda w: nys.QKPrepare(2, 1, 64, q_weight=w, k_weight=w, rotation=rotation, device=dev)
    w = torch.full((64,), 2.0, device=dev)
    want = make(w).rows(x, None, pos, torch.empty_like(x))[0]
    torch.cuda.synchronize()
    return torch, x, pos, w, want, make


def test_made_on_one_stream_used_on_another(cuda_device):
    torch, x, pos, w, want, make = _set(cuda_device)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        old = [torch.full((64,), -3.0, device=cuda_device) for _ in range(8)]
        del old                                  # what the copies' memory holds before they are made
        torch.cuda._sleep(WAIT)
        prep = make(w * 1.0)
    out = torch.empty_like(x)
    with torch.cuda.stream(b):
        prep.rows(x, None, pos, out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_dropped_while_a_call_is_queued(cuda_device):
    torch, x, pos, w, want, make = _set(cuda_device)
    b = torch.cuda.Stream()
    prep, out = make(w), torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(b):
        torch.cuda._sleep(WAIT)
        prep.rows(x, None, pos, out)
    del prep
    new = [torch.full((64,), -3.0, device=cuda_device) for _ in range(64)]
    torch.cuda.current_stream().synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(new) == 64
