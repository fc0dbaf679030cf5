"""f32 layers of infinities, NaN and values above bf16's largest: on every kernel, results are infinite, NaN or finite as
those of the f32 products are, and the finite ones within the bounds of test_gpu_layers."""
import numpy as np
import pytest

from differentiable_gaussian_splatting_amd import binding as B
from tests.layer_calls import CALLS
from tests.test_gpu_layers import _t, close, ctx, product_bound, u  # noqa: F401

pytestmark = pytest.mark.gpu

INF, HUGE = float("inf"), 3.4e38   # f32's largest is 3.4028e38, bf16's 3.3895e38
HUGE32 = float(np.float32(HUGE))
# few rows and narrow ones, every f32 tile whole, split and mixed, values one by one
SIZES = [(5, 200, 130), (40, 300, 70), (300, 32, 48), (300, 3, 200)] + [c[2:] for c in CALLS if c[1] == "f32" and c[0] == "fwd"]
BACKWARD = [(300, 32, 48), (300, 3, 200)] + [c[2:] for c in CALLS if c[1] == "f32" and c[0] == "bwd"]


def spoil(x, at=0):
    """Places of every kind, in rows `at` to `at` + 4."""
    n, k = x.shape
    x[at % n, k // 2] = INF
    x[(at + 1) % n, -1] = -INF
    x[(at + 2) % n, 0] = HUGE
    x[(at + 3) % n, 0], x[(at + 3) % n, k - 1] = INF, -INF
    x[(at + 4) % n, k // 3] = float("nan")
    return x


def compare(got, want, bound, either=None):
    """either: places where a product is beyond f32 and another infinite, where NaN and infinity are both f32's answer
    (it depends on whether the product is rounded by itself, and on the order)."""
    torch = _t()
    over = want.isfinite() & (want.abs() > torch.finfo(torch.float32).max)
    want = torch.where(over, want.sign() * INF, want)
    fine = want.isfinite()
    assert torch.equal(got.isfinite(), fine)
    sure = torch.ones_like(fine) if either is None else ~either
    assert torch.equal(got.isnan()[sure], want.isnan()[sure])
    assert torch.equal(got[want.isinf() & sure].double(), want[want.isinf() & sure])
    close(got[fine], want[fine], bound[fine])


def product(a, b):
    """a b^T in f64, its bound, and the places where a finite product is beyond f32 beside infinite ones."""
    torch = _t()
    z = a @ b.T
    beyond = torch.zeros_like(z, dtype=torch.bool)
    for r, c in (a.abs() == HUGE32).nonzero().tolist():
        beyond[r] |= (a[r, c] * b[:, c]).abs() > torch.finfo(torch.float32).max
    for r, c in (b.abs() == HUGE32).nonzero().tolist():
        beyond[:, r] |= (b[r, c] * a[:, c]).abs() > torch.finfo(torch.float32).max
    return z, product_bound("f32", a.shape[1], a, b), beyond & ~z.isfinite()


@pytest.mark.parametrize("n,k,f", SIZES)
def test_forward(ctx, n, k, f):
    torch = _t()
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = spoil(torch.randn((n, k), generator=g, device="cuda"), seed * 3)
        w = torch.randn((f, k), generator=g, device="cuda") * k ** -0.5
        if seed:
            w[4 % f, k // 2], w[7 % f] = INF, 0.0
        z, e, either = product(x.double(), w.double())
        compare(B.gs_linear_fwd(ctx, x, w), z, e + 2 * u * z.abs(), either)
        z = z.clamp(min=0)
        compare(B.gs_linear_fwd(ctx, x, w, act="relu"), z, e + 2 * u * z.abs(), either)
        pre = torch.empty((n, f - f % 2), device="cuda")
        B.gs_gated_fwd(ctx, x, w[:f - f % 2], act="none", pre=pre)
        z, e, either = product(x.double(), w[:f - f % 2].double())
        compare(pre, z, e + 2 * u * z.abs(), either)


@pytest.mark.parametrize("n,k,f", BACKWARD)
def test_gradients(ctx, n, k, f):
    torch = _t()
    g = torch.Generator(device="cuda").manual_seed(7)
    for places in range(3):
        x, w = torch.randn((n, k), generator=g, device="cuda"), torch.randn((f, k), generator=g, device="cuda") * f ** -0.5
        d = torch.randn((n, f), generator=g, device="cuda") * 0.01
        for t in (x, w, d)[places:places + 1]:
            spoil(t, 2)
        if places == 2:
            d[3, 0] = 0.0
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        B.gs_linear_bwd(ctx, x, w, d, dx=dx, dw=dw)
        want, e, either = product(d.double(), w.double().T)
        compare(dx, want, e + 2 * u * want.abs(), either)
        want, e, either = product(d.double().T, x.double().T)
        compare(dw, want, e + 2 * u * want.abs(), either)
