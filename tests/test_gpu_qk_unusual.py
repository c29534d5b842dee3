"""Rows whose squares fp32 does not hold: what the header says comes of them, and nothing of
their neighbours."""
import math

import pytest

pytestmark = pytest.mark.gpu

# d, rot, interleaved: pairs within a lane, of neighbours, across lanes, none
FORMS = [(64, 64, False), (128, 128, True), (80, 52, False), (64, 0, False)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 1e30])
def test_rows_past_fp32(cuda_device, dtype, value, form):
    import torch
    from streaming_nystr_landmark_gb300 import nys
    dt, dev, (d, rot, inter) = getattr(torch, dtype), cuda_device, form
    if value == 1e30 and dtype == "float16":
        value = math.inf
    g = torch.Generator(device=dev).manual_seed(1)
    rotation = nys.Rotation(d, rot=rot, interleaved=inter, device=dev) if rot else None
    prep = nys.QKPrepare(2, 1, d, dtype=dt, q_weight=torch.full((d,), 1.25, device=dev), rotation=rotation, device=dev)
    x = torch.randn((3, 2, d), generator=g, device=dev).to(dt)
    pos = torch.tensor([1, 2, 3], dtype=torch.int32, device=dev)
    clean = prep.rows(x, None, pos, torch.empty_like(x))[0]
    x[1, 0, 5] = value
    out = prep.rows(x, None, pos, torch.empty_like(x))[0]
    assert torch.equal(out[[0, 2]], clean[[0, 2]]) and torch.equal(out[1, 1], clean[1, 1])
    row = out[1, 0]
    if math.isnan(value):
        assert bool(row.isnan().all())
    elif math.isinf(value):
        mine = [5] if not rot else [5, 4] if inter else [5, 5 + rot // 2]
        others = [i for i in range(d) if i not in mine]
        assert bool(row[mine].isnan().all()) and not bool(row[others].any())
    else:
        assert not bool(row.any())
