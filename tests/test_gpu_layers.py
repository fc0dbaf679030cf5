"""Linear and gated layers with their gradients, and the Muon update, against
the formulas in 64 bits.

u = 2^-24 is the rounding error of f32, U that of the output type, T that of
the layer's type; the bounds below were fixed before the kernels ran:
* a sum of K products in f32, in any order and with each addition off by at
  most 2u (matrix instructions need not round to nearest): 2 (K + 2) u sum |x w|;
  f32 factors are held in parts: 2^-22 |x w| more for each product;
* activations: slopes are at most 1.13 (gelu's largest), their evaluation is
  within 16 u (1 + |z|) (a dozen roundings; |z| sigma(v) sigma(-v) |v| < |z|);
* their slopes: within 16 u (1 + |z|) as well, |z sigma' v'| < 2 |z| included;
* dz rounded to the layer's type: T |dz| per factor of the gradients;
* one rounding of the output: U |out|.
"""
import ctypes as C
import math

import pytest

from differentiable_gaussian_splatting_amd import binding as B
from tests.test_gpu_tensors import UNIT, dtype, rows_view

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu", "sigmoid"]
# rows, in, out; extra columns between rows, values before the first
SHAPES = [(1, 1, 1, 0, 0), (1, 64, 48, 0, 0), (3, 5, 2, 1, 1), (16, 300, 33, 0, 0), (17, 31, 65, 3, 1),
          (257, 35, 64, 0, 0), (130, 129, 127, 7, 5), (500, 32, 48, 27, 0), (128, 256, 128, 0, 0), (1000, 1, 3, 0, 0),
          (65, 1030, 70, 0, 1), (2, 2051, 515, 1, 0), (300, 260, 300, 4, 4)]


def _t():
    import torch
    return torch


@pytest.fixture(scope="module")
def ctx():
    assert _t().cuda.is_available(), "GPU tests need a GPU"
    c = B.Context()
    yield c
    c.close()


def close(got, want, bound):
    """|got - want| <= bound, all in f64 on the device."""
    torch = _t()
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), float(err[bad].max()), float((err / bound)[bad].max()))


def untouched(view, base_before):
    """Nothing of the view's buffer changed but the view."""
    torch = _t()
    mask = torch.ones_like(base_before, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert torch.equal(view._base[mask], base_before[mask])


def value_and_slope(z, act):
    torch = _t()
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    k = 2.0 * math.sqrt(2.0 / math.pi)
    v = k * (z + 0.044715 * z ** 3) if act == "gelu" else z
    dv = k * (1 + 3 * 0.044715 * z ** 2) if act == "gelu" else torch.ones_like(z)
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    return (p, p * q) if act == "sigmoid" else (z * p, p + z * p * q * dv)


def unit(name):
    return UNIT[name]


def product_bound(name, k, a, b):
    """Error of a b^T over k values, a and b in f64."""
    each = 2 * (k + 2) * u + (2.0 ** -22 if name == "f32" else 0.0)
    return each * (a.abs() @ b.abs().T) + 1e-37


def case(n, k, f, name, extra=0, lead=0, seed=0):
    x = rows_view(n, k, name, extra, lead, seed=seed + 1)
    w = rows_view(f, k, name, extra, lead, seed=seed + 2, scale=max(k, 1) ** -0.5)
    return x, w


def check_fwd(ctx, n, k, f, name, act, extra=0, lead=0, bias=None, residual=None, pre=False, out=None, gated=False):
    torch = _t()
    x, w = case(n, k, f * (2 if gated else 1), name, extra, lead)
    b = None if bias is None else torch.randn(f, device="cuda").to(dtype(bias))
    r = None if residual is None else rows_view(n, f, residual, extra, lead, seed=9)
    o = rows_view(n, f, out or name, extra, lead, seed=5)
    p = rows_view(n, f * (2 if gated else 1), name, extra, lead, seed=6) if pre else None
    before, pbefore = o._base.clone(), p._base.clone() if pre else None
    if gated:
        B.gs_gated_fwd(ctx, x, w, act=act, pre=p, out=o)
    else:
        B.gs_linear_fwd(ctx, x, w, bias=b, act=act, residual=r, pre=p, out=o)
    X, W = x.double(), w.double()
    z, ez = X @ W.T, product_bound(name, k, X, W)
    if b is not None:
        ez = ez + u * (z.abs() + ez + b.double().abs())
        z = z + b.double()
        ez = ez + u * z.abs()
    T, tiny_t = unit(name)
    if pre:
        close(p, z, ez + T * (z.abs() + ez) + tiny_t)
        untouched(p, pbefore)
    if gated:
        g, up, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
        a = value_and_slope(g, act)[0]
        ea = 1.13 * eg + 16 * u * (1 + g.abs())
        y = a * up
        ey = ea * (up.abs() + eu) + a.abs() * eu + u * y.abs()
    else:
        y = value_and_slope(z, act)[0]
        ey = ez if act == "none" else 1.13 * ez + 16 * u * (1 + z.abs())
        if r is not None:
            y = y + r.double()
            ey = ey + u * (y.abs() + ey)
    U, tiny = unit(out or name)
    close(o, y, ey + U * (y.abs() + ey) + tiny)
    untouched(o, before)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,f,extra,lead", SHAPES)
def test_linear(ctx, n, k, f, extra, lead, name):
    act = ACTS[(n + k + f) % 5]
    check_fwd(ctx, n, k, f, name, act, extra, lead)
    check_fwd(ctx, n, k, f, name, "none", extra, lead, bias="f32", residual=name, pre=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_linear_activations(ctx, name, act):
    check_fwd(ctx, 70, 40, 50, name, act, bias=name, pre=True)
    check_fwd(ctx, 70, 40, 50, name, act, 2, 1, bias="f32", residual="f32", pre=True, out="f32")
    check_fwd(ctx, 3, 700, 130, name, act, bias="f32", residual=name)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,f,extra,lead", SHAPES)
def test_gated(ctx, n, k, f, extra, lead, name):
    check_fwd(ctx, n, k, f, name, "silu", extra, lead, pre=True, gated=True)
    check_fwd(ctx, n, k, f, name, ACTS[(n + f) % 5], extra, lead, gated=True, out="f32")


def test_large_products(ctx):
    """Several tiles of every kind in each direction, with and without splits of the inner length."""
    for name in ("f32", "bf16"):
        check_fwd(ctx, 1100, 520, 900, name, "gelu", bias="f32", pre=True)
        check_fwd(ctx, 300, 4100, 400, name, "none", 3, 1, residual=name)
        check_fwd(ctx, 1100, 300, 700, name, "silu", pre=True, gated=True)
        check_bwd(ctx, 1100, 520, 900, name, "silu", bias="f32")
        check_bwd(ctx, 5000, 70, 130, name, "relu", 1, 1, bias=name)
    check_fwd(ctx, 2600, 192, 2200, "f16", "relu", bias="f16", pre=True)
    check_bwd(ctx, 2600, 300, 2200, "f16", "gelu")


# ---------------------------------------------------------------------------- gradients

def check_bwd(ctx, n, k, f, name, act, extra=0, lead=0, bias=None, accumulate=False, gated=False, dw="same",
              dout="same", want_dx=True):
    torch = _t()
    dw, dout = (name if t == "same" else t for t in (dw, dout))
    both = f * (2 if gated else 1)
    x, w = case(n, k, both, name, extra, lead)
    z = rows_view(n, both, name, extra, lead, seed=3)
    d = rows_view(n, f, dout, extra, lead, seed=4)
    gx = rows_view(n, k, name, extra, lead, seed=6) if want_dx else None
    gw = rows_view(both, k, dw, extra, lead, seed=7)
    gb = None if bias is None else torch.randn(both, device="cuda").to(dtype(bias))
    bx, bw = gx._base.clone() if want_dx else None, gw._base.clone()
    old_w, old_b = gw.double() if accumulate else 0.0, gb.double() if accumulate and gb is not None else 0.0
    if gated:
        B.gs_gated_bwd(ctx, x, w, z, d, act=act, dx=gx, dw=gw, accumulate=accumulate)
    else:
        B.gs_linear_bwd(ctx, x, w, d, pre=z if act != "none" else None, act=act, dx=gx, dw=gw, dbias=gb,
                        accumulate=accumulate)
    X, W, Z, D = x.double(), w.double(), z.double(), d.double()
    T, tiny_t = unit(name)
    if gated:
        g, up = Z[:, :f], Z[:, f:]
        a, s = value_and_slope(g, act)
        ea = 16 * u * (1 + g.abs())
        dz = torch.cat([D * up * s, D * a], 1)
        e = torch.cat([(D * up).abs() * (ea + 2 * u * s.abs()), D.abs() * (ea + u * a.abs())], 1)
    else:
        s = value_and_slope(Z, act)[1]
        dz = D * s
        e = torch.zeros_like(dz) if act == "none" else D.abs() * 16 * u * (1 + Z.abs()) + u * dz.abs()
    rounded = e if act == "none" and not gated and dout == name else e + T * (dz.abs() + e) + tiny_t
    if want_dx:
        want = dz @ W
        ex = product_bound(name, both, dz.abs() + rounded, W.T) + rounded @ W.abs()
        close(gx, want, ex + T * (want.abs() + ex) + tiny_t)
        untouched(gx, bx)
    U, tiny = unit(dw)
    want = dz.T @ X + old_w
    ew = product_bound(name, n, dz.abs().T + rounded.T, X.T) + rounded.T @ X.abs()
    ew = ew + u * (want.abs() + ew)
    close(gw, want, ew + U * (want.abs() + ew) + tiny)
    untouched(gw, bw)
    if gb is not None:
        Ub, tb = unit(bias)
        want = dz.sum(0) + old_b
        eb = ((n + 2) * u * (dz.abs() + e) + e).sum(0)
        eb = eb + u * (want.abs() + eb)
        close(gb, want, eb + Ub * (want.abs() + eb) + tb)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,f,extra,lead", SHAPES)
def test_linear_gradient(ctx, n, k, f, extra, lead, name):
    check_bwd(ctx, n, k, f, name, "none", extra, lead, bias="f32", dw="f32")
    check_bwd(ctx, n, k, f, name, ACTS[1 + (n + k + f) % 4], extra, lead, bias=name)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_linear_gradient_activations(ctx, name, act):
    check_bwd(ctx, 90, 45, 70, name, act, bias="f32", accumulate=True, dw="f32", dout="f32")
    check_bwd(ctx, 90, 45, 70, name, act, 1, 1, want_dx=False)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,f,extra,lead", SHAPES)
def test_gated_gradient(ctx, n, k, f, extra, lead, name):
    check_bwd(ctx, n, k, f, name, "silu", extra, lead, gated=True)
    check_bwd(ctx, n, k, f, name, ACTS[(n + f) % 5], extra, lead, gated=True, accumulate=True, dw="f32", dout="f32")


@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 127, 129])
@pytest.mark.parametrize("k,f", [(63, 65), (64, 64), (128, 31), (33, 129), (16, 16)])
def test_sizes_around_the_tiles(ctx, n, k, f):
    for name in ("f32", "bf16"):
        check_fwd(ctx, n, k, f, name, "silu", bias="f32", pre=True)
        check_bwd(ctx, n, k, f, name, "silu", bias="f32")
        check_fwd(ctx, n, k, f, name, "gelu", gated=True)


@pytest.mark.parametrize("n", [1, 20, 64, 65])
def test_few_rows_accumulate(ctx, n):
    for name in ("f32", "bf16"):
        check_bwd(ctx, n, 300, 333, name, "silu", bias="f32", accumulate=True, dw="f32")
        check_bwd(ctx, n, 300, 333, name, "none", bias=name, accumulate=True)
        check_bwd(ctx, n, 40, 24, name, "gelu", bias=name, accumulate=True)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,f", [(3, 70, 40), (40, 130, 72), (300, 260, 300), (129, 200, 136), (1000, 64, 48), (700, 7, 5),
                                   (2100, 72, 2056)])
def test_nothing_around_the_operands_is_read(ctx, n, k, f, name):
    """Views into buffers of NaN: gaps between rows (aligned ones and others), before the first and behind the last."""
    torch = _t()

    def view(rows, cols, gap, lead):
        ld = cols + gap
        buf = torch.full((lead + rows * ld + 64,), float("nan"), device="cuda").to(dtype(name))
        v = buf.as_strided((rows, cols), (ld, 1), lead)
        v.copy_(torch.randn((rows, cols), device="cuda"))
        return v

    for gap, lead in ((8 - k % 8, 8), (3, 1)):
        x, w, d, z = view(n, k, gap, lead), view(f, k, gap, lead), view(n, f, 8, lead), view(n, f, 8, lead)
        b, out = torch.zeros(f, device="cuda"), torch.empty((n, f), device="cuda")
        dx, dw, db = torch.empty_like(x), torch.empty((f, k), device="cuda"), torch.empty(f, device="cuda")
        X, W, D = x.double(), w.double(), d.double()
        B.gs_linear_fwd(ctx, x, w, bias=b, out=out)
        e = product_bound(name, k, X, W)
        close(out, X @ W.T, e + 2 * u * ((X @ W.T).abs() + e))
        for act in ("none", "relu"):
            B.gs_linear_bwd(ctx, x, w, d, pre=z, act=act, dx=dx, dw=dw, dbias=db)
            dz = D if act == "none" else D * (z > 0)   # exact in every type
            e = product_bound(name, n, dz.T, X.T)
            close(dw, dz.T @ X, e + 2 * u * ((dz.T @ X).abs() + e))
            e = product_bound(name, f, dz, W.T)
            T, tiny = unit(name)
            close(dx, dz @ W, e + T * ((dz @ W).abs() + e) + tiny)
            close(db, dz.sum(0), (n + 2) * u * dz.abs().sum(0) + 1e-37)
        if f % 2 == 0:
            y = torch.empty((n, f // 2), device="cuda")
            B.gs_gated_fwd(ctx, x, w, act="none", out=y)
            Z, ez = X @ W.T, product_bound(name, k, X, W)
            g, q = Z[:, :f // 2], Z[:, f // 2:]
            eg, eq = ez[:, :f // 2], ez[:, f // 2:]
            bound = eg * q.abs() + eq * g.abs() + eg * eq
            close(y, g * q, bound + 2 * u * ((g * q).abs() + bound))


def test_layers_of_nothing(ctx):
    torch = _t()
    x, w = torch.randn((5, 4), device="cuda"), torch.randn((6, 4), device="cuda")
    b = torch.randn(6, device="cuda")
    assert B.gs_linear_fwd(ctx, x[:0], w, bias=b).shape == (0, 6)
    assert B.gs_linear_fwd(ctx, x, w[:0]).shape == (5, 0)
    # without inputs the product is zero
    out = B.gs_linear_fwd(ctx, x[:, :0], w[:, :0], bias=b, residual=torch.ones((5, 6), device="cuda"))
    assert torch.equal(out, (b + 1.0).expand(5, 6))
    assert torch.equal(B.gs_gated_fwd(ctx, x[:, :0], w[:, :0]), torch.zeros((5, 3), device="cuda"))
    dw, db, dx = torch.ones((6, 4), device="cuda"), torch.ones(6, device="cuda"), torch.ones((5, 4), device="cuda")
    B.gs_linear_bwd(ctx, x[:0], w, torch.empty((0, 6), device="cuda"), dw=dw, dbias=db, accumulate=True)
    assert torch.equal(dw, torch.ones_like(dw)) and torch.equal(db, torch.ones_like(db))
    B.gs_linear_bwd(ctx, x[:0], w, torch.empty((0, 6), device="cuda"), dw=dw, dbias=db)
    assert not dw.any() and not db.any()
    B.gs_linear_bwd(ctx, x, w[:0], torch.empty((5, 0), device="cuda"), dx=dx)
    assert not dx.any()
    B.gs_linear_bwd(ctx, x, w, torch.empty((5, 6), device="cuda"))   # nothing wanted


def test_broadcast_and_in_place(ctx):
    """One row read for all of x; a residual that is the output."""
    torch = _t()
    for name in ("f32", "bf16"):
        t = dtype(name)
        x, w = torch.randn((1, 40), device="cuda").to(t), torch.randn((24, 40), device="cuda").to(t)
        wide = B.gs_linear_fwd(ctx, x.expand(70, 40), w)
        one = B.gs_linear_fwd(ctx, x.expand(70, 40).contiguous(), w)
        assert torch.equal(wide, one)
        for n in (1, 70, 300):
            x = torch.randn((n, 2000), device="cuda").to(t)
            w = torch.randn((24, 2000), device="cuda").to(t)
            r = torch.randn((n, 24), device="cuda").to(t)
            want = B.gs_linear_fwd(ctx, x, w, act="gelu", residual=r)
            got = B.gs_linear_fwd(ctx, x, w, act="gelu", residual=r, out=r)
            assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_special_values_stay_in_their_rows(ctx, name):
    """A NaN or an infinity in a row of x changes that row alone (also behind the last whole tile), and one in a
    masked place of dout (its pre at -inf) only what the formula says."""
    torch = _t()
    t = dtype(name)
    for n, k, f in ((5, 70, 40), (200, 33, 66), (140, 300, 130)):
        x, w = torch.randn((n, k), device="cuda").to(t), torch.randn((f, k), device="cuda").to(t)
        clean = B.gs_linear_fwd(ctx, x, w, act="silu")
        y = x.clone()
        y[1, k - 1], y[3, 0] = float("nan"), float("inf")
        got = B.gs_linear_fwd(ctx, y, w, act="silu")
        keep = [i for i in range(n) if i not in (1, 3)]
        assert torch.equal(got[keep], clean[keep]) and got[1].isnan().all()
        if name != "f32":
            assert not got[3].isfinite().all()
        # activations at the ends of the range: no NaN from infinities
        z = torch.tensor([float("-inf"), float("inf"), -3e38 if name != "f16" else -6e4, 0.0], device="cuda").to(t)
        eye = torch.zeros((4, 4), device="cuda").to(t)
        for act, want in (("relu", [0.0, math.inf]), ("silu", [0.0, math.inf]), ("gelu", [0.0, math.inf]),
                          ("sigmoid", [0.0, 1.0])):
            out = B.gs_linear_fwd(ctx, eye, eye, bias=z, act=act)
            assert out[0, :2].tolist() == want, act
            d = torch.zeros(4, device="cuda")
            B.gs_linear_bwd(ctx, eye, eye, torch.ones((1, 4), device="cuda").to(t).expand(4, 4), pre=z.expand(4, 4),
                            act=act, dbias=d)
            slopes = {"sigmoid": [0.0, 0.0]}.get(act, [0.0, 4.0])
            assert d[:2].tolist() == slopes and d.isfinite().all(), act


def test_offsets_past_32_bits(ctx):
    """An x of 4.7e9 values: its last rows, and the gradient of a w that only they reach."""
    torch = _t()
    n, k, f = 72_000, 65_536, 8
    x = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((f, k), dtype=torch.bfloat16, device="cuda")
    x[-1, -1], x[-2, 0], x[-2, -3] = 3.0, 5.0, 2.0
    w[:, -1], w[2, 0], w[3, -3] = 2.0, 1.0, 0.5
    out = B.gs_linear_fwd(ctx, x, w)
    want = torch.zeros((n, f), device="cuda")
    want[-1], want[-2, 2], want[-2, 3] = 6.0, 5.0, 1.0
    assert torch.equal(out.float(), want)
    d = torch.zeros((n, f), dtype=torch.bfloat16, device="cuda")
    d[-1, 1], d[-2, 4] = 4.0, 8.0
    dw = torch.empty_like(w)
    dx = torch.empty_like(x)
    B.gs_linear_bwd(ctx, x, w, d, dw=dw, dx=dx)
    want = torch.zeros((f, k), device="cuda")
    want[1, -1], want[4, 0], want[4, -3] = 12.0, 40.0, 16.0
    assert torch.equal(dw.float(), want)
    assert torch.equal(dx[-2:].float(), torch.stack([d[-2].float() @ w.float(), d[-1].float() @ w.float()]))
    assert not dx[:-2].any()


def test_more_columns_than_a_grid_has_threads_for(ctx):
    """One row into 2^28 + 5 columns, and the bias gradient of 2^30 + 70."""
    torch = _t()
    f = (1 << 28) + 5
    w = torch.ones((f, 1), dtype=torch.bfloat16, device="cuda")
    w[-1], w[-7], w[1 << 20] = 3.0, -2.0, 0.5
    x = torch.full((1, 1), 4.0, dtype=torch.bfloat16, device="cuda")
    out = B.gs_linear_fwd(ctx, x, w)
    assert torch.equal(out.view(-1), w.view(-1) * 4)
    del w, out
    f = (1 << 30) + 70
    w = torch.empty((f, 0), dtype=torch.bfloat16, device="cuda")
    d = torch.ones((1, f), dtype=torch.bfloat16, device="cuda")
    d[0, -1], d[0, 5] = 3.0, -1.0
    db = torch.zeros(f, dtype=torch.bfloat16, device="cuda")
    B.gs_linear_bwd(ctx, x[:, :0], w, d, dbias=db)
    assert torch.equal(db, d.view(-1))


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_tiles_that_end_with_their_operands(ctx, name):
    """Last tiles moved back: every output is written once (a residual in place would be added twice), also where some
    tiles are split over k and some are not, at every kind of alignment."""
    torch = _t()
    t = dtype(name)
    for n, k, f in ((129, 200, 130), (257, 72, 264), (700, 1000, 513), (321, 64, 2056), (1000, 520, 1001)):
        x, w = torch.randn((n, k), device="cuda").to(t), (torch.randn((f, k), device="cuda") * k ** -0.5).to(t)
        r = torch.randn((n, f), device="cuda")
        want = r.double() + x.double() @ w.double().T
        X, W = x.double(), w.double()
        B.gs_linear_fwd(ctx, x, w, residual=r, out=r)
        e = product_bound(name, k, X, W)
        close(r, want, e + 3 * u * (want.abs() + e))
        d = torch.randn((n, f), device="cuda").to(t)
        dw = torch.randn((f, k), device="cuda")
        want = dw.double() + d.double().T @ X
        B.gs_linear_bwd(ctx, x, w, d, dw=dw, accumulate=True)
        e = product_bound(name, n, d.double().T, X.T)
        close(dw, want, e + 3 * u * (want.abs() + e))
        # rows further apart than they are long, from an address that is not a multiple of 16
        check_fwd(ctx, n, k, f, name, "silu", 8, 0, bias="f32", pre=True)
        check_fwd(ctx, n, k, f, name, "relu", 3, 1, pre=True, gated=True)
        check_bwd(ctx, n, k, f, name, "gelu", 8, 0, bias="f32")


@pytest.mark.parametrize("act", ACTS[2:])
def test_gradients_are_those_of_the_layers(ctx, act):
    """Derivatives along random directions against differences of the forward pass, linear then gated then linear,
    f32.  The loss is a sum in f64; its differences over 2 h with h = 1/64 are off by h^2 / 6 times a third derivative
    (a few units here: 2e-4) and by the forward pass's errors over h (1e-5 * 64 = 6e-4), against derivatives of about
    one: 2e-2 of the larger of 1 and the derivative is allowed."""
    torch = _t()
    g = torch.Generator().manual_seed(5)
    R = lambda *s: (torch.randn(*s, generator=g)).cuda()
    n = 40
    x, w1, b1, w2, w3 = R(n, 20), R(30, 20) * 0.2, R(30) * 0.1, R(2 * 26, 30) * 0.2, R(12, 26) * 0.2
    c = R(n, 12) / n ** 0.5

    def forward(x, w1, b1, w2, w3, keep=None):
        p1, p2 = torch.empty((n, 30), device="cuda"), torch.empty((n, 52), device="cuda")
        h1 = B.gs_linear_fwd(ctx, x, w1, bias=b1, act=act, pre=p1)
        h2 = B.gs_gated_fwd(ctx, h1, w2, act=act, pre=p2)
        if keep is not None:
            keep += [p1, h1, p2, h2]
        y = B.gs_linear_fwd(ctx, h2, w3)
        return float((y.double() * c.double()).sum())

    keep = []
    forward(x, w1, b1, w2, w3, keep)
    p1, h1, p2, h2 = keep
    dw3, dh2, dw2, dh1 = torch.empty_like(w3), torch.empty_like(h2), torch.empty_like(w2), torch.empty_like(h1)
    dw1, db1, dx = torch.empty_like(w1), torch.empty_like(b1), torch.empty_like(x)
    B.gs_linear_bwd(ctx, h2, w3, c, dx=dh2, dw=dw3)
    B.gs_gated_bwd(ctx, h1, w2, p2, dh2, act=act, dx=dh1, dw=dw2)
    B.gs_linear_bwd(ctx, x, w1, dh1, pre=p1, act=act, dx=dx, dw=dw1, dbias=db1)
    h = 1.0 / 64
    for i, (t, d) in enumerate(((x, dx), (w1, dw1), (b1, db1), (w2, dw2), (w3, dw3))):
        v = R(*t.shape)
        v /= v.norm()
        args = [x, w1, b1, w2, w3]
        both = []
        for sign in (h, -h):
            args[i] = t + sign * v
            both.append(forward(*args))
        want, got = (both[0] - both[1]) / (2 * h), float((d.double() * v.double()).sum())
        assert abs(got - want) <= 2e-2 * max(1.0, abs(want)), (i, got, want)


# ---------------------------------------------------------------------------- Muon

COEF = (3.4445, -4.7750, 2.0315)


def newton_schulz(v, steps, extra_norm=0.0):
    """The definition in 64 bits, and a bound on the Frobenius norm of the f32 evaluation's error.

    With e the error of X, s the shorter side, l the longer one and spectral norms |X| <= 1.21, |G| <= 1.47,
    |P| <= 2.81: G's error is 2 |X| e plus its own rounding, (2 l u + 3 2^-22) |X|_F^2; P's |b| + 2 |c| |G| times
    that, plus (2 s u + 3 2^-22) |c| |G|_F^2 + 3 u |b| |G|_F; the new X's
    e + (a + |P|) e + |X| P's + (2 s u + 3 2^-22) |P|_F |X|_F + 3 u a |X|_F, times 1.01 for products of errors.  The
    first-order amplification of e itself is that of the polynomial map on matrices, at most its largest divided
    difference on [0, 1.21], which is a = 3.4445 at 0 (its slope lies in [-1.6, 3.4445]), whatever the terms above
    add up to: the terms in e are replaced by 3.4445 e."""
    torch = _t()
    a, b, c = COEF
    X = v / (v.norm() + 1e-7)
    e = 8 * u + 2 * extra_norm
    tall = v.shape[0] > v.shape[1]
    s, l = min(v.shape), max(v.shape)
    part = 3 * 2.0 ** -22
    for _ in range(steps):
        G = X.T @ X if tall else X @ X.T
        P = b * G + c * (G @ G)
        own_g = (2 * l * u + part) * float(X.norm()) ** 2
        own_p = (abs(b) + 2 * c * 1.47) * own_g + (2 * s * u + part) * c * float(G.norm()) ** 2 + \
            3 * u * abs(b) * float(G.norm())
        e = 1.01 * (a * e + 1.21 * own_p + (2 * s * u + part) * float(P.norm()) * float(X.norm()) +
                    3 * u * a * float(X.norm()))
        X = a * X + (X @ P if tall else P @ X)
    return X, e


def check_muon(ctx, shapes, name="f32", nesterov=True, decay=0.01, steps=5, copy=None, extra=0, lead=0, norm=None,
               momentum=0.95, lr=0.02, scale=0.01):
    torch = _t()
    gen = torch.Generator().manual_seed(len(shapes) + sum(r * 7 + c for r, c in shapes))
    R = lambda r, c, s: (torch.randn((r, c), generator=gen) * s).cuda()
    p, m = [R(r, c, 0.05) for r, c in shapes], [R(r, c, scale) for r, c in shapes]
    g = [rows_view(r, c, name, extra, lead, seed=k, scale=scale) for k, (r, c) in enumerate(shapes)]
    q = None if copy is None else [torch.zeros(s, dtype=dtype(copy), device="cuda") for s in shapes]
    old = [(a.double(), b.double()) for a, b in zip(p, m)]
    B.gs_muon_tensors(ctx, p, m, g, lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=decay, steps=steps,
                      norm=norm, copies=q)
    f = 1.0 if norm is None else float(norm[1])
    for k, (r, c) in enumerate(shapes):
        if r * c == 0:
            continue
        P0, M0 = old[k]
        G = f * g[k].double()
        mu = float(torch.tensor(momentum, dtype=torch.float32))
        M1 = mu * M0 + G
        size = M0.abs() + G.abs()
        close(m[k], M1, 4 * u * size + 1e-44)
        U = G + mu * M1 if nesterov else M1
        off = float((8 * u * size).norm() / max(float(U.norm()), 1e-30))   # of u, relative
        X, e = newton_schulz(U, steps, off)
        rate = lr * max(1.0, r / c) ** 0.5
        want = (1.0 - lr * decay) * P0 - rate * X
        err = float((p[k].double() - want).norm())
        bound = rate * e + 4 * u * float(P0.norm() + rate * X.norm()) + 1e-37
        assert err <= bound, (k, r, c, err, bound)
        if q is not None:
            assert torch.equal(q[k], p[k].to(q[k].dtype))


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (33, 20), (48, 64), (64, 48), (64, 64),
                                   (65, 64), (100, 300), (129, 127), (128, 515), (600, 130), (257, 260)])
def test_muon(ctx, shape):
    check_muon(ctx, [shape])
    check_muon(ctx, [shape], name="bf16", nesterov=False, decay=0.0, copy="f16", extra=3, lead=1)


@pytest.mark.parametrize("steps", [0, 1, 2, 12])
def test_muon_steps(ctx, steps):
    # the rounding bound grows 3.4445-fold a step: at 12 it says little, but all stays finite
    check_muon(ctx, [(40, 24), (130, 200)], steps=steps)


def test_muon_lists(ctx):
    mixed = [(64, 48), (0, 5), (48, 64), (7, 300), (300, 7), (5, 0), (200, 140), (1, 64), (64, 64)]
    check_muon(ctx, mixed, copy="bf16")
    check_muon(ctx, [(8 + k % 5, 6 + k % 7) for k in range(105)], name="f16")
    check_muon(ctx, [])


def test_muon_of_large_matrices(ctx):
    """Every tile, products split over the long side, more matrices than a launch takes, both orientations."""
    check_muon(ctx, [(1100, 900), (513, 2000)], copy="bf16")
    check_muon(ctx, [(2300, 70), (64, 5000)], name="bf16")
    check_muon(ctx, [(150, 140 + k % 3) for k in range(50)] + [(130 + k % 2, 190) for k in range(49)], steps=3)
    check_muon(ctx, [(2048, 1536)], steps=2)
    check_muon(ctx, [(3, 1000), (1000, 3), (1, 4000)])


def test_muon_in_more_than_one_group(ctx):
    """2.01e8 values: two groups, one after the other in the same workspace."""
    torch = _t()
    n = 8192
    p = [torch.zeros((n, n), device="cuda") for _ in range(3)]
    m = [torch.zeros((n, n), device="cuda") for _ in range(3)]
    g = [torch.randn((n, n), device="cuda") for _ in range(3)]
    B.gs_muon_tensors(ctx, p, m, g, lr=-1.0, steps=2, momentum=0.0)
    for k in (0, 2):
        X, e = newton_schulz(g[k].double(), 2, 2 * u)
        assert torch.equal(m[k], g[k])
        assert float((p[k].double() - X).norm()) <= e + 4 * u * float(X.norm())
        del X


def test_muon_of_zero_and_tiny_gradients(ctx):
    torch = _t()
    p, m, g = (torch.zeros((20, 30), device="cuda") for _ in range(3))
    p += 1.5
    B.gs_muon_tensors(ctx, [p], [m], [g])
    assert torch.equal(p, torch.full_like(p, 1.5)) and not m.any()
    check_muon(ctx, [(20, 30), (90, 70)], scale=1e-9)     # beside the epsilon
    check_muon(ctx, [(20, 30), (90, 70)], scale=1e18)     # squares beyond f32
    # one value alone: its place has the Frobenius norm
    m.zero_()
    p.zero_()
    g[3, 4] = -2.0
    B.gs_muon_tensors(ctx, [p], [m], [g], lr=1.0)
    assert (p != 0).sum() == 1 and 0.6 < float(p[3, 4]) < 1.25


def test_muon_takes_the_clip_factor_and_leaves_steps_out(ctx):
    torch = _t()
    norm = torch.tensor([4.0, 0.25], device="cuda")
    check_muon(ctx, [(30, 50), (70, 64)], norm=norm)
    p, m, g = (torch.randn((30, 20), device="cuda") for _ in range(3))
    q = torch.zeros_like(p)
    keep = [t.clone() for t in (p, m)]
    for bad in (float("nan"), float("inf")):
        norm = torch.tensor([bad, 0.0], device="cuda")
        B.gs_muon_tensors(ctx, [p], [m], [g], norm=norm, copies=[q])
        assert torch.equal(p, keep[0]) and torch.equal(m, keep[1]) and not q.any()
    # a value that is not finite spoils its own matrix only
    g2 = g.clone()
    g[0, 0] = float("nan")
    p2, m2 = p.clone(), m.clone()
    p3, m3 = p.clone(), m.clone()
    B.gs_muon_tensors(ctx, [p, p2], [m, m2], [g, g2])
    B.gs_muon_tensors(ctx, [p3], [m3], [g2])
    assert p.isnan().all() and torch.equal(p2, p3) and torch.equal(m2, m3)


# ---------------------------------------------------------------------------- together

class Net:
    """Features from a table through linear, gated and linear layers; matrices updated by Muon, the rest by Adam."""

    def __init__(self, n=700, rows=50, t="f32", seed=0):
        torch = _t()
        g = torch.Generator().manual_seed(seed)
        R = lambda *s: torch.randn(*s, generator=g).cuda()
        self.idx = torch.randint(0, rows, (n,), generator=g).int().cuda()
        self.table, self.w = R(rows, 32), [R(64, 32) * 0.2, R(2 * 96, 64) * 0.1, R(48, 96) * 0.1]
        self.b = [R(64) * 0.1, R(48) * 0.1]
        self.target = R(n, 48)
        E = lambda *s: torch.empty(s, device="cuda")
        self.x, self.p1, self.h1, self.p2, self.h2, self.y = E(n, 32), E(n, 64), E(n, 64), E(n, 192), E(n, 96), E(n, 48)
        self.dx, self.dh1, self.dh2, self.dtable = E(n, 32), E(n, 64), E(n, 96), torch.empty_like(self.table)
        self.dw, self.db = [torch.empty_like(w) for w in self.w], [torch.empty_like(b) for b in self.b]
        self.m = [torch.zeros_like(w) for w in self.w]
        self.am, self.av = ([torch.zeros_like(t) for t in [self.table] + self.b] for _ in range(2))
        self.norm = torch.zeros(2, device="cuda")

    def state(self):
        return [self.table] + self.w + self.b + self.m + self.am + self.av + [self.norm, self.y]

    def forward(self, c):
        B.gs_embed_fwd(c, self.table, self.idx, self.x)
        B.gs_linear_fwd(c, self.x, self.w[0], bias=self.b[0], act="silu", pre=self.p1, out=self.h1)
        B.gs_gated_fwd(c, self.h1, self.w[1], act="gelu", pre=self.p2, out=self.h2)
        B.gs_linear_fwd(c, self.h2, self.w[2], bias=self.b[1], out=self.y)

    def step(self, c, k=1, dy=None):
        self.forward(c)
        dy = (self.y - self.target) / self.y.numel() if dy is None else dy
        B.gs_linear_bwd(c, self.h2, self.w[2], dy, dx=self.dh2, dw=self.dw[2], dbias=self.db[1])
        B.gs_gated_bwd(c, self.h1, self.w[1], self.p2, self.dh2, act="gelu", dx=self.dh1, dw=self.dw[1])
        B.gs_linear_bwd(c, self.x, self.w[0], self.dh1, pre=self.p1, act="silu", dx=self.dx, dw=self.dw[0],
                        dbias=self.db[0])
        B.gs_embed_bwd(c, self.idx, self.dx, self.dtable)
        B.gs_grad_norm(c, self.dw + self.db + [self.dtable], 1.0, self.norm)
        B.gs_muon_tensors(c, self.w, self.m, self.dw, norm=self.norm)
        B.gs_adam_tensors(c, [self.table] + self.b, self.am, self.av, [self.dtable] + self.db, step=k, norm=self.norm)


def test_a_network_trains_and_agrees_with_autograd(ctx):
    torch = _t()
    net = Net()
    net.step(ctx)
    # the gradients against those of the same network in f64 (h, p: f32 roundings only, so 1e-4 of the norm is
    # a thousand times their size: sums of at most 700 terms, u sqrt(700) each)
    net = Net()
    leaves = [t.double().requires_grad_() for t in [net.table] + net.w + net.b]
    table, w0, w1, w2, b0, b1 = leaves
    h = torch.nn.functional.silu(table[net.idx.long()] @ w0.T + b0)
    z = h @ w1.T
    h = torch.nn.functional.gelu(z[:, :96], approximate="tanh") * z[:, 96:]
    y = h @ w2.T + b1
    (0.5 * (y - net.target.double()) ** 2).mean().backward()
    net.step(ctx)
    for got, leaf in zip([net.dtable] + net.dw + net.db, leaves):
        assert float((got.double() - leaf.grad).norm()) <= 1e-4 * float(leaf.grad.norm())
    for k in range(2, 5):
        net.step(ctx, k)
    assert all(t.isfinite().all() for t in net.state())


def test_a_scene_whose_colours_come_from_a_network(ctx):
    """Lookup, linear, gated and linear layers make a view's SH rows; the view's gradient rows go back through them
    as they lie (columns of wider rows), and every update runs."""
    torch = _t()
    from differentiable_gaussian_splatting_amd import scenes
    w = scenes.make_workload("c3_gmm4k", n=700, width=96, height=64, seed=3)
    ds = B.DeviceScene(w.scene, "cuda")
    assert ds.sh.numel() == 700 * 48
    target = torch.from_numpy(w.target).cuda()
    net = Net(n=700, seed=4)
    net.forward(ctx)
    ds.sh.view(700, 48).copy_(0.2 * net.y)
    rows = torch.zeros((700, 59), device="cuda")
    B.gs_train_view(ctx, w.camera, ds, target, grad3d_out=rows)
    assert rows[:, 11:].any()
    keep = net.y.clone()
    net.step(ctx, dy=rows[:, 11:])
    assert torch.equal(net.y, keep)
    d = rows[:, 11:].double()
    want = d.T @ net.h2.double()
    e = 2 * (700 + 2) * u * (d.abs().T @ net.h2.double().abs())
    close(net.dw[2], want, e + u * (want.abs() + e) + 1e-37)
    assert all(t.isfinite().all() for t in net.state()) and net.m[0].any()


def test_results_repeat_and_streams(ctx):
    """The same bits on another stream, with other work beside it, as on the context's."""
    torch = _t()
    a, b = Net(seed=1), Net(seed=1)
    s = torch.cuda.Stream()
    c = B.Context(stream=s)
    s.wait_stream(torch.cuda.current_stream())
    for k in range(1, 4):
        a.step(ctx, k)
        with torch.cuda.stream(s):
            b.step(c, k)
    torch.cuda.synchronize()
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)
    c.close()


def test_graph_replays(ctx):
    torch = _t()
    stream = torch.cuda.Stream()
    c = B.Context(stream=stream)
    net = Net(seed=2)
    big = [torch.randn((300, 3000), device="cuda").bfloat16(), torch.randn((130, 3000), device="cuda").bfloat16()]
    out, dw = torch.empty((300, 130), device="cuda"), torch.empty((130, 3000), device="cuda")
    d, db = torch.randn((300, 130), device="cuda"), torch.empty(130, device="cuda")
    pre = torch.empty((300, 130), device="cuda").bfloat16()

    def step(cc):
        net.step(cc)
        B.gs_linear_fwd(cc, big[0], big[1], act="gelu", pre=pre, out=out)
        B.gs_linear_bwd(cc, big[0], big[1], d, pre=pre, act="gelu", dw=dw, dbias=db)

    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(c)
    for rep in range(4):
        net.idx.copy_(torch.randint(0, 50, net.idx.shape))
        big[0].normal_()
        keep = [t.clone() for t in net.state()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in net.state() + [out, dw, db, pre]]
        for t, k in zip(net.state(), keep):
            t.copy_(k)
        step(ctx)
        torch.cuda.synchronize()
        for x, y in zip(got, net.state() + [out, dw, db, pre]):
            assert torch.equal(x, y), rep
    c.close()


def test_allocation_failure_leaves_outputs(ctx):
    torch = _t()
    from tests.test_gpu_errors import FailingContext
    f = FailingContext()
    x, w = torch.randn((300, 2000), device="cuda"), torch.randn((70, 2000), device="cuda")
    z, d = torch.randn((300, 70), device="cuda"), torch.randn((300, 70), device="cuda")
    outs = [torch.full(s, 7.0, device="cuda") for s in ((300, 70), (300, 2000), (70, 2000), (70,))]
    p, m = torch.full((70, 90), 7.0, device="cuda"), torch.full((70, 90), 7.0, device="cuda")
    g = torch.randn((70, 90), device="cuda")
    live = f.mem_stats()["live"]
    for call in (lambda: B.gs_linear_fwd(f, x, w, out=outs[0]),
                 lambda: B.gs_linear_bwd(f, x, w, d, pre=z, act="silu", dx=outs[1], dw=outs[2], dbias=outs[3]),
                 lambda: B.gs_muon_tensors(f, [p], [m], [g])):
        k, same = 1, [t.clone() for t in outs + [p, m]]
        while True:
            f.arm(k)
            try:
                call()
                break
            except B.GsError as e:
                assert e.status == B.GS_ERR_OOM
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(same, outs + [p, m])) and f.mem_stats()["live"] == live
            k += 1
        f.arm(0)
        assert f.mem_stats()["live"] == live
    f.close()


# ---------------------------------------------------------------------------- refusals

def refused(status, fn):
    with pytest.raises(B.GsError) as e:
        fn()
    assert e.value.status == status


def test_refusals(ctx):
    torch = _t()
    bad = B.GS_ERR_INVALID_ARG
    R = lambda *s: torch.randn(*s, device="cuda")
    x, w, out, b = R(4, 6), R(8, 6), R(4, 8), R(8)
    lin = lambda **kw: B.gs_linear_fwd(ctx, kw.pop("x", x), kw.pop("w", w), **{"out": out, **kw})
    for kw in (dict(out=out[:3]), dict(out=out[:, :7]), dict(w=R(8, 5)), dict(w=w.half()), dict(x=x.half()),
               dict(out=out[:1].expand(4, 8)), dict(bias=b[:7]), dict(bias=R(8, 1)), dict(residual=R(4, 7)),
               dict(bias=b.half()), dict(pre=out.half()), dict(pre=R(3, 8)), dict(out=out.half())):
        refused(bad, lambda: lin(**kw))
    with pytest.raises(ValueError):
        lin(act="tanh")
    with pytest.raises(ValueError):
        lin(x=x.cpu())
    with pytest.raises(ValueError):
        lin(w=R(6, 8).t())
    bwd = lambda **kw: B.gs_linear_bwd(ctx, x, w, kw.pop("d", out), **{"pre": out, "act": "silu", **kw})
    for kw in (dict(pre=None), dict(pre=R(4, 7)), dict(d=R(3, 8)), dict(dx=R(4, 5)), dict(dw=R(8, 5)),
               dict(dx=x.half()), dict(dbias=R(7)), dict(dw=w[:1].expand(8, 6)), dict(d=out.half())):
        refused(bad, lambda: bwd(**kw))
    refused(bad, lambda: B.gs_gated_fwd(ctx, x, w[:7], out=R(4, 3)))
    refused(bad, lambda: B.gs_gated_fwd(ctx, x, w, out=out))
    refused(bad, lambda: B.gs_gated_fwd(ctx, x, w, pre=R(4, 4), out=R(4, 4)))
    refused(bad, lambda: B.gs_gated_bwd(ctx, x, w, R(4, 4), R(4, 4), dx=R(4, 6)))
    muon = lambda **kw: B.gs_muon_tensors(ctx, kw.pop("p", [R(4, 6)]), kw.pop("m", [R(4, 6)]), kw.pop("g", [R(4, 6)]), **kw)
    for kw in (dict(steps=-1), dict(steps=21), dict(momentum=1.0), dict(momentum=-0.1), dict(lr=float("nan")),
               dict(weight_decay=float("inf")), dict(p=[R(4, 6).half()]), dict(m=[R(6, 4)]), dict(g=[R(4, 5)]),
               dict(p=[R(4, 8)[:, :6]]), dict(copies=[R(4, 5).half()])):
        refused(bad, lambda: muon(**kw))
    with pytest.raises(ValueError):
        muon(g=[])
    with pytest.raises(ValueError):
        muon(norm=torch.empty(1, device="cuda"))


def test_refusals_at_the_c_entries(ctx):
    L, h = ctx.lib, ctx.handle
    torch = _t()
    x = torch.randn((4, 6), device="cuda")
    T = lambda **kw: B.gs_tensor(*[{**dict(data=x.data_ptr(), rows=4, cols=6, stride=6, type=0, pad=0), **kw}[k]
                                   for k in ("data", "rows", "cols", "stride", "type", "pad")])
    bad, over = B.GS_ERR_INVALID_ARG, B.GS_ERR_OVERFLOW
    ok, sq = C.byref(T()), C.byref(T(cols=4))
    for t, st in ((T(type=3), bad), (T(rows=-1), bad), (T(data=0), bad), (T(data=x.data_ptr() + 1), bad),
                  (T(rows=1 << 41, stride=0), over), (T(rows=1 << 31, cols=1, stride=0), over)):
        assert L.gs_linear_fwd(h, C.byref(t), ok, None, 0, None, None, sq) == st
        assert L.gs_linear_fwd(h, ok, C.byref(t), None, 0, None, None, sq) == st
        assert L.gs_last_error(h)
    for act in (-1, 5):
        assert L.gs_linear_fwd(h, ok, ok, None, act, None, None, sq) == bad
        assert L.gs_gated_fwd(h, ok, ok, act, None, sq) == bad
    assert L.gs_linear_fwd(None, ok, ok, None, 0, None, None, sq) == bad
    for k in range(3):
        args = [ok, ok, sq]
        args[k] = None
        assert L.gs_linear_fwd(h, args[0], args[1], None, 0, None, None, args[2]) == bad
        assert L.gs_linear_bwd(h, args[0], args[1], None, 0, args[2], 0, None, None, None) == bad
    assert L.gs_gated_bwd(h, ok, ok, None, 2, C.byref(T(cols=2)), 0, None, None) == bad
    q = C.cast(C.pointer(T()), C.c_void_p)
    o = B.gs_muon_opts(5, 1, 0.02, 0.95, 0.0)
    assert L.gs_muon_tensors(h, q, q, q, None, 1, None, None) == bad
    assert L.gs_muon_tensors(h, None, q, q, None, 1, C.byref(o), None) == bad
    assert L.gs_muon_tensors(h, q, q, q, None, -1, C.byref(o), None) == bad
    assert L.gs_muon_tensors(None, q, q, q, None, 1, C.byref(o), None) == bad
    wide = C.cast(C.pointer(T(rows=1, cols=(1 << 20) + 1, stride=0)), C.c_void_p)
    assert L.gs_muon_tensors(h, wide, wide, wide, None, 1, C.byref(o), None) == over
