"""Gradients of 16-bit layers where dz = dout act'(pre), or dout times the other half of a gated layer, leaves f16's
range (2^-24 to 65504), as a scaled loss in f32 makes it: against the formulas in 64 bits.

u, T, U and the bounds are those of test_gpu_layers.  f16 values of dz are scaled by a power of two before they are
rounded.  The call's scale brings its largest finite |dz| to at least 2^14, so that rounding is off by T |dz| or, below
f16's normal range, by half a step of 2^-24 there: 2^-25 / 2^14 = 2^-39 of that largest.  dx takes it too where every
row's largest is at least 2^-14 of the call's, 1 after scaling, and what is lost 2^-25 of the row's largest at most;
else each row has a scale of its own, and 2^-39.
"""
import pytest

from differentiable_gaussian_splatting_amd import binding as B
from tests.test_gpu_layers import _t, close, ctx, product_bound, u, unit, value_and_slope  # noqa: F401
from tests.test_gpu_tensors import dtype

pytestmark = pytest.mark.gpu

# rows, in, out: narrow layers in one pass, both products in one launch, tiles of every kind, splits over k
SIZES = [(300, 40, 48), (33, 128, 16), (1, 64, 64), (5, 70, 300), (200, 260, 300), (257, 1000, 131), (2000, 24, 600),
         (4100, 520, 520)]


def gradients(ctx, n, k, f, name, gated, dout, act="silu", wscale=1.0, change=None, seed=0, dw_type=None):
    """dx, dw (f32 unless dw_type) and what the bounds need."""
    torch = _t()
    g = torch.Generator(device="cuda").manual_seed(seed + n + k + f)
    R = lambda *s: torch.randn(s, generator=g, device="cuda")
    t, both = dtype(name), f * (2 if gated else 1)
    x, w, z = R(n, k).to(t), (R(both, k) * (wscale * k ** -0.5)).to(t), R(n, both).to(t)
    d = R(n, f) * dout
    if change is not None:
        change(x, d)
    dx, dw = torch.empty_like(x), torch.empty((both, k), device="cuda", dtype=dw_type or torch.float32)
    if gated:
        B.gs_gated_bwd(ctx, x, w, z, d, act=act, dx=dx, dw=dw)
    else:
        B.gs_linear_bwd(ctx, x, w, d, pre=z, act=act, dx=dx, dw=dw)
    Z, D = z.double(), d.double()
    if gated:
        a, s = value_and_slope(Z[:, :f], act)
        up, ea = Z[:, f:], 16 * u * (1 + Z[:, :f].abs())
        dz = torch.cat([D * up * s, D * a], 1)
        e = torch.cat([(D * up).abs() * (ea + 2 * u * s.abs()), D.abs() * (ea + u * a.abs())], 1)
    else:
        dz = D * value_and_slope(Z, act)[1]
        e = D.abs() * 16 * u * (1 + Z.abs()) + u * dz.abs()
    return dx, dw, x.double(), w.double(), dz, e


def check(name, dx, dw, X, W, dz, e, rows=slice(None), only_dx=False):
    """dx of `rows`, and dw."""
    n, both = dz.shape
    T, tiny = unit(name)
    off = e + T * (dz.abs() + e)
    by_row = off + (2.0 ** -25 if name == "f16" else 0.0) * dz.abs().amax(1, keepdim=True)
    want = dz @ W
    ex = product_bound(name, both, dz.abs() + by_row, W.T) + by_row @ W.abs()
    bound = ex + T * (want.abs() + ex) + tiny
    # dx is of the layer's type: what rounds beyond its largest is infinite, of the value's sign
    most = _t().finfo(dx.dtype).max
    over = want.abs() - bound > most * (1 + T)
    may = ~over & (want.abs() + bound > most)
    assert (dx[rows][over[rows]].double() == want[rows][over[rows]].sign() * float("inf")).all()
    inside = ~over & ~(may & dx.isinf())
    close(_t().where(inside, dx.double(), want)[rows], want[rows], bound[rows])
    if only_dx:
        return
    off = off + (2.0 ** -39 if name == "f16" else 0.0) * dz.abs().max()
    want = dz.T @ X
    ew = product_bound(name, n, (dz.abs() + off).T, X.T) + off.T @ X.abs()
    close(dw, want, ew + u * (want.abs() + ew) + 1e-37)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,k,f", SIZES)
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_dz_beyond_the_range_of_f16(ctx, name, n, k, f, gated):
    # dx of about wscale dout: within f16
    for dout, wscale in ((1e7, 1e-4), (3e20, 2.0 ** -24), (1.0, 1.0), (1e-9, 1e4), (1e-30, 1e4)):
        check(name, *gradients(ctx, n, k, f, name, gated, dout, wscale=wscale))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,k,f", SIZES)
def test_rows_of_different_sizes_do_not_meet(ctx, n, k, f, gated):
    """dx of rows beside ones that are larger by 1e25, infinite or NaN; dw of rows within 1e10 of each other, or 0."""
    torch = _t()

    def spoil(x, d):
        d[::3] *= 1e25
        d[1::7, 0] = float("nan")
        d[2::7, -1] = float("inf")

    keep = torch.ones(n, dtype=torch.bool)
    keep[::3] = keep[1::7] = keep[2::7] = False
    r = gradients(ctx, n, k, f, "f16", gated, 1.0, change=spoil)
    dz, e = (torch.where(keep[:, None].cuda(), t, torch.zeros_like(t)) for t in r[4:])
    check("f16", r[0], r[1], r[2], r[3], dz, e, rows=keep.cuda(), only_dx=True)

    for big in (1e5, 30.0, 0.0):   # beyond and within what one scale for all rows holds; masked rows
        def spread(x, d):
            d[::2] /= big if big else 1.0
            d[::5] *= big

        check("f16", *gradients(ctx, n, k, f, "f16", gated, 1.0, change=spread, wscale=1e-2))


def test_dout_of_the_layers_type_and_no_activation(ctx):
    """f32 dout without an activation is rounded for the products as dz is; f16 dout of a gated layer grows by u."""
    torch = _t()
    for n, k, f in ((200, 260, 300), (70, 40, 48)):
        check("f16", *gradients(ctx, n, k, f, "f16", False, 1e8, act="none", wscale=1e-5))
        x, w = torch.randn((n, k), device="cuda").half(), torch.randn((2 * f, k), device="cuda").half() * 0.001
        z, d = torch.full((n, 2 * f), 300.0, device="cuda").half(), torch.full((n, f), 1000.0, device="cuda").half()
        dx, dw = torch.empty_like(x), torch.empty((2 * f, k), device="cuda")
        B.gs_gated_bwd(ctx, x, w, z, d, act="none", dx=dx, dw=dw)
        D = torch.full((n, 2 * f), 300000.0, device="cuda", dtype=torch.float64)
        check("f16", dx, dw, x.double(), w.double(), D, 2 * u * D)


def test_one_gradient_alone_and_accumulated(ctx):
    torch = _t()
    n, k, f = 150, 300, 200
    x, w, z = (torch.randn(s, device="cuda").half() for s in ((n, k), (f, k), (n, f)))
    d = torch.randn((n, f), device="cuda") * 1e6
    w *= 1e-3
    dx, dw, db = torch.empty_like(x), torch.empty((f, k), device="cuda"), torch.empty(f, device="cuda")
    B.gs_linear_bwd(ctx, x, w, d, pre=z, act="gelu", dx=dx, dw=dw, dbias=db)
    assert dx.isfinite().all() and dw.isfinite().all()
    dx2, dw2, dw3, db2 = torch.empty_like(dx), torch.empty_like(dw), dw.clone(), torch.empty_like(db)
    B.gs_linear_bwd(ctx, x, w, d, pre=z, act="gelu", dx=dx2)
    B.gs_linear_bwd(ctx, x, w, d, pre=z, act="gelu", dw=dw2)
    B.gs_linear_bwd(ctx, x, w, d, pre=z, act="gelu", dbias=db2)
    B.gs_linear_bwd(ctx, x, w, d, pre=z, act="gelu", dw=dw3, accumulate=True)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2) and torch.equal(dw3, 2 * dw)


def test_graph_whose_rows_come_to_differ(ctx):
    """Replays on values of other sizes: rows that share a scale, then rows that need their own, then masked ones."""
    torch = _t()
    n, k, f = 300, 264, 136
    stream = torch.cuda.Stream()
    c = B.Context(stream=stream)
    x, w, z = (torch.randn(s, device="cuda").half() for s in ((n, k), (2 * f, k), (n, 2 * f)))
    d, dx, dw = torch.randn((n, f), device="cuda"), torch.empty_like(x), torch.empty((2 * f, k), device="cuda")
    go = lambda cc: B.gs_gated_bwd(cc, x, w, z, d, dx=dx, dw=dw)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        go(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        go(c)
    for rep, (some, others) in enumerate(((1.0, 1.0), (1e-9, 10.0), (1e-30, 1e-28), (0.0, 1.0), (1.0, 1e20))):
        d.normal_()
        d[::2] *= some
        d[1::2] *= others
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = dx.clone(), dw.clone()
        dx.fill_(7.0)
        dw.fill_(7.0)
        go(ctx)
        torch.cuda.synchronize()
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and dw.isfinite().all(), rep
    c.close()


def test_allocation_failure_leaves_f16_gradients(ctx):
    torch = _t()
    from tests.test_gpu_errors import FailingContext
    c = FailingContext()
    x, w, z = (torch.randn(s, device="cuda").half() for s in ((300, 200), (2 * 70, 200), (300, 2 * 70)))
    d = torch.randn((300, 70), device="cuda")
    dx, dw = torch.full((300, 200), 7.0, device="cuda").half(), torch.full((2 * 70, 200), 7.0, device="cuda")
    live, k = c.mem_stats()["live"], 1
    while True:
        c.arm(k)
        try:
            B.gs_gated_bwd(c, x, w, z, d, dx=dx, dw=dw)
            break
        except B.GsError as e:
            assert e.status == B.GS_ERR_OOM
            torch.cuda.synchronize()
            assert (dx == 7).all() and (dw == 7).all() and c.mem_stats()["live"] == live
        k += 1
    assert k > 3
    c.arm(0)
    c.close()
