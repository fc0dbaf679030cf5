"""What gs_kernel_time counts for the layer calls: the launches that there were."""
import pytest

from differentiable_gaussian_splatting_amd import binding as B
from tests.test_gpu_layers import _t

pytestmark = pytest.mark.gpu

NAMES = ("layer_few", "layer_narrow", "layer_mm", "layer_dz", "layer_sum", "muon")


def test_only_launches_are_counted():
    torch = _t()
    c = B.Context()
    B.gs_set_timing(c, True)
    R = lambda *s: torch.randn(s, device="cuda")

    def counts(call):
        B.gs_reset_timing(c)
        call()
        return {n: k for n in NAMES for ms, k in [B.gs_kernel_time(c, n)] if k}

    # k, f and t: few rows, narrow rows, tiles (one too wide for the narrow kernels by its outputs, one by its inputs)
    for name in (torch.float32, torch.float16, torch.bfloat16):
        for n, k, f, want in ((5, 300, 200, "layer_few"), (500, 32, 48, "layer_narrow"), (500, 300, 200, "layer_mm"),
                              (500, 16, 400, "layer_mm"), (500, 1000, 16, "layer_mm")):
            x, w = R(n, k).to(name), R(f, k).to(name)
            assert counts(lambda: B.gs_linear_fwd(c, x, w)) == {want: 1}, (name, n, k, f)
            assert counts(lambda: B.gs_gated_fwd(c, x, w)) == {want: 1}, (name, n, k, f)
    x, w, z = R(500, 300), R(200, 300), R(500, 200)
    dx, dw, db = R(500, 300), R(200, 300), R(200)
    assert counts(lambda: B.gs_linear_bwd(c, x, w, z, pre=z, act="silu", dx=dx)) == {"layer_dz": 1, "layer_mm": 1}
    x, w, z, dw = R(500, 32), R(48, 32), R(500, 48), R(48, 32)
    assert counts(lambda: B.gs_linear_bwd(c, x, w, z, dw=dw)) == {"layer_narrow": 1, "layer_sum": 1}
    assert counts(lambda: B.gs_muon_tensors(c, [w], [R(48, 32)], [dw])) == {"muon": 1}
    B.gs_set_timing(c, False)
    c.close()
