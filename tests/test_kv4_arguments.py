"""Arguments of the Python classes that stand for no number, without a GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
nys = pytest.importorskip("streaming_nystr_landmark_gb300.nys")


@pytest.mark.parametrize("base", [0, 0.0, -1.0, -10000.0, math.inf, math.nan, 1e-320])
def test_bases_that_give_no_frequencies(base):
    with pytest.raises(ValueError):
        nys.Rotation(64, base=base, device="cpu")


def test_frequencies_need_no_base():
    assert nys.Rotation(4, base=0, freqs=[1.0, 0.5], device="cpu").turns.shape == (2,)
    assert nys.Rotation(4, base=0, rot=0, device="cpu").turns.shape == (0,)
    assert nys.Rotation(4, base=0.5, device="cpu").turns.shape == (2,)


@pytest.mark.parametrize("scale", [1e-46, 1e-300, 1e39, 1e308])
def test_scales_that_f32_does_not_hold(scale):
    """0 would be taken for 1/sqrt(d)."""
    with pytest.raises(ValueError, match="scale"):
        nys.ExactAttention(2, 1, 64, 64, scale=scale, device="cpu")
