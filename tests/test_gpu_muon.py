"""The Muon update at the ends of f32's range."""
import pytest

from differentiable_gaussian_splatting_amd import binding as B  # noqa: F401
from tests.test_gpu_layers import _t, check_muon, ctx  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [0, 1])
def test_norms_beyond_the_largest_float(ctx, steps):
    """|u| of 3e39 to 6e40, whose inverse is no normal float; a large lr, so that the update outweighs the parameters."""
    check_muon(ctx, [(60, 40), (300, 200), (1100, 900)], scale=3e37, steps=steps, lr=1e4, decay=0.0)
