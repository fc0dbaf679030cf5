"""Table lookup and its gradient, the global gradient norm with clipping, and
Adam over tensor lists, against the formulas in 64 bits.

u = 2^-24 is the rounding error of f32, U that of the output type; the bounds
below count the roundings of the f32 evaluation and were fixed before the
kernels ran:
* lookup: one product and one rounding: (u + U) |x|;
* table gradient: k values added in f32 in any order: (k + 1) u sum |x|, one
  product with the scale, one rounding (and, accumulating, one sum);
* norm and factor: f64 sums rounded once, 2u; clipped values: the factor's 2u,
  a product, a rounding: (4u + U) |x|;
* Adam: see _adam_bounds.
"""
import ctypes as C
import math

import numpy as np
import pytest

from differentiable_gaussian_splatting_amd import binding as B

pytestmark = pytest.mark.gpu

u = 2.0 ** -24


def _t():
    import torch
    return torch


@pytest.fixture(scope="module")
def ctx():
    assert _t().cuda.is_available(), "GPU tests need a GPU"
    c = B.Context()
    yield c
    c.close()


def dtype(name):
    torch = _t()
    return dict(f32=torch.float32, f16=torch.float16, bf16=torch.bfloat16, i32=torch.int32, i64=torch.int64)[name]


# relative rounding error and half the smallest subnormal of each type
UNIT = dict(f32=(2.0 ** -24, 2.0 ** -150), f16=(2.0 ** -11, 2.0 ** -25), bf16=(2.0 ** -8, 2.0 ** -134))


def rows_view(n, w, name, extra=0, lead=0, seed=0, scale=1.0):
    """An n x w matrix whose rows are `extra` values apart beyond their width
    and whose first value is `lead` values into its buffer."""
    torch = _t()
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn(lead + n * (w + extra) + extra, generator=g) * scale).to(dtype(name)).cuda()
    return buf[lead:].as_strided((n, w), (w + extra, 1), lead)


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, bound):
    got, want = f64(got), np.asarray(want)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), err[bad].max(), np.broadcast_to(bound, err.shape)[bad][err[bad].argmax()])


def sample_index(n, v, kind, seed=0):
    rng = np.random.default_rng(seed)
    if v == 0:
        return rng.integers(-3, 4, n)
    i = dict(uniform=lambda: rng.integers(0, v, n), one=lambda: np.full(n, v // 2),
             distinct=lambda: rng.permutation(max(n, v))[:n] % v, sorted=lambda: np.sort(rng.integers(0, v, n)),
             zipf=lambda: (np.exp(rng.random(n) * math.log(v + 1)).astype(np.int64) - 1) * 7 % v,
             hot=lambda: np.where(rng.random(n) < 0.6, v - 1, rng.integers(0, v, n)),
             masked=lambda: np.where(rng.random(n) < 0.4, rng.choice([-1, v, v + 5, -2 ** 31, 2 ** 31 - 1], n),
                                     rng.integers(0, v, n)),
             none=lambda: np.full(n, -1))[kind]()
    return i.astype(np.int64)


# ---------------------------------------------------------------------------- lookup

@pytest.mark.parametrize("index", ["i32", "i64"])
@pytest.mark.parametrize("types", ["f32-f32", "bf16-bf16", "f16-f16", "bf16-f32", "f32-f16"])
@pytest.mark.parametrize("n,v,w,extra,lead", [(1, 1, 1, 0, 0), (1, 7, 4096, 0, 0), (5, 3, 2, 1, 1), (64, 100, 48, 0, 0),
                                              (257, 33, 45, 14, 3), (1000, 17, 3, 0, 0), (33, 50, 1027, 5, 1),
                                              (129, 9, 64, 8, 8), (300, 11, 513, 0, 1)])
def test_lookup(ctx, n, v, w, extra, lead, types, index):
    torch = _t()
    tn, on = types.split("-")
    table = rows_view(v, w, tn, extra, lead, seed=n + w)
    idx = torch.from_numpy(sample_index(n, v, "masked" if n > 1 else "uniform", n)).to(dtype(index)).cuda()
    out = rows_view(n, w, on, extra, lead, seed=5)
    before = out._base.clone()
    scale = 0.40625
    B.gs_embed_fwd(ctx, table, idx, out, scale=scale)
    i = idx.cpu().numpy()
    inside = (i >= 0) & (i < v)
    want = np.where(inside[:, None], f64(table)[np.clip(i, 0, v - 1)] * scale, 0.0)
    U, tiny = UNIT[on]
    close(out, want, (u + U) * np.abs(want) + tiny)
    # nothing but out's own values is written
    after = out._base.clone()
    mask = torch.ones_like(after, dtype=torch.bool)
    mask.as_strided((n, w), out.stride(), lead).fill_(False)
    assert torch.equal(after[mask], before[mask])


def test_lookup_without_scale_is_a_copy_and_keeps_special_values(ctx):
    torch = _t()
    for name in ("f32", "f16", "bf16"):
        table = torch.randn(6, 37).to(dtype(name)).cuda()
        table[1, 3], table[2, 5], table[3, 7] = float("nan"), float("inf"), -0.0
        idx = torch.tensor([[1, 3], [2, -1]], device="cuda")
        out = B.gs_embed_fwd(ctx, table, idx)
        assert out.shape == (4, 37) and out.dtype == table.dtype
        want = torch.cat([table[1:2], table[3:4], table[2:3], torch.zeros_like(table[:1])])
        assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(out.isnan(), want.isnan())
        assert math.copysign(1.0, float(out[1, 7])) == -1.0


def test_lookup_of_nothing(ctx):
    torch = _t()
    table = torch.randn(4, 8, device="cuda")
    assert B.gs_embed_fwd(ctx, table, torch.empty(0, dtype=torch.int64, device="cuda")).shape == (0, 8)
    assert B.gs_embed_fwd(ctx, table[:, :0], torch.zeros(3, dtype=torch.int64, device="cuda")).shape == (3, 0)
    # a table without rows: every index is outside it
    out = B.gs_embed_fwd(ctx, table[:0], torch.tensor([0, 1, -1], device="cuda"))
    assert torch.equal(out, torch.zeros(3, 8, device="cuda"))


def test_offsets_past_32_bits(ctx):
    """A table of 4.8e9 values: lookup of its last rows, and its gradient."""
    torch = _t()
    v, w = 75_000, 64_000
    table = torch.zeros((v, w), dtype=torch.bfloat16, device="cuda")
    table[-1], table[-2] = 3.0, 5.0
    idx = torch.tensor([v - 1, 0, v - 2], device="cuda")
    out = B.gs_embed_fwd(ctx, table, idx, scale=2.0)
    assert out[0].eq(6.0).all() and out[1].eq(0.0).all() and out[2].eq(10.0).all()
    table.fill_(1.0)
    B.gs_embed_bwd(ctx, idx, out, table, scale=0.5)
    assert table[-1].eq(3.0).all() and table[-2].eq(5.0).all() and float(table[:-2].float().abs().max()) == 0.0
    # gradient rows 2^31 values apart
    far = torch.zeros(2 * (1 << 31) + 16, dtype=torch.bfloat16, device="cuda").as_strided((3, 16), (1 << 31, 1))
    far[0], far[1], far[2] = 1.0, 2.0, 4.0
    d = torch.empty((2, 16), device="cuda")
    B.gs_embed_bwd(ctx, torch.tensor([1, 0, 1], device="cuda"), far, d)
    assert d[0].eq(2.0).all() and d[1].eq(5.0).all()


def test_output_of_more_than_one_launch_row(ctx):
    """36e9 values of bf16: more packs than a launch has threads in x."""
    torch = _t()
    n, w = 1_100_000, 32_768
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 72 GB of free device memory")
    table = torch.zeros((3, w), dtype=torch.bfloat16, device="cuda")
    table[1], table[2] = 1.0, 2.0
    idx = (torch.arange(n, device="cuda") % 3).int()
    out = torch.empty((n, w), dtype=torch.bfloat16, device="cuda")
    B.gs_embed_fwd(ctx, table, idx, out)
    for a in range(0, n, 100_000):
        part = out[a:a + 100_000]
        want = idx[a:a + 100_000].float()
        assert torch.equal(part.amax(1).float(), want) and torch.equal(part.amin(1).float(), want)
    del out
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------- its gradient

def table_gradient(i, x, v, padding):
    """sum, sum of magnitudes and count of each row, in 64 bits"""
    keep = (i >= 0) & (i < v) & (i != padding)
    s, a, k = np.zeros((v, x.shape[1])), np.zeros((v, x.shape[1])), np.zeros(v)
    np.add.at(s, i[keep], x[keep])
    np.add.at(a, i[keep], np.abs(x[keep]))
    np.add.at(k, i[keep], 1.0)
    return s, a, k


def check_gradient(ctx, n, v, w, kind, tn="f32", on="f32", index="i32", extra=0, lead=0, padding=-1,
                   accumulate=False, scale=0.40625):
    torch = _t()
    i = sample_index(n, v, kind, n + v)
    dout = rows_view(n, w, tn, extra, lead, seed=n + w)
    idx = torch.from_numpy(i).to(dtype(index)).cuda()
    dtable = rows_view(v, w, on, extra, lead, seed=9)
    old, whole = f64(dtable), dtable._base.clone()
    B.gs_embed_bwd(ctx, idx, dout, dtable, scale=scale, padding=padding, accumulate=accumulate)
    s, a, k = table_gradient(i, f64(dout), v, padding)
    want = s * scale + (old if accumulate else 0.0)
    U, tiny = UNIT[on]
    bound = (k[:, None] + 2.0) * u * a * abs(scale) + (U + 2 * u) * np.abs(want) + tiny
    if accumulate:
        bound += u * np.abs(old)
        bound[k == 0] = 0.0
    close(dtable, want, bound)
    after = dtable._base.clone()
    mask = torch.ones_like(after, dtype=torch.bool)
    mask.as_strided((v, w), dtable.stride(), lead).fill_(False)
    assert torch.equal(after[mask], whole[mask])
    # the same bits again
    first = dtable.clone()
    whole2 = whole.clone()
    again = whole2.as_strided((v, w), dtable.stride(), lead)
    B.gs_embed_bwd(ctx, idx, dout, again, scale=scale, padding=padding, accumulate=accumulate)
    assert torch.equal(again, first)


@pytest.mark.parametrize("kind", ["uniform", "one", "distinct", "sorted", "zipf", "hot", "masked", "none"])
@pytest.mark.parametrize("n,v,w", [(1, 1, 1), (2, 5, 3), (63, 7, 48), (257, 1000, 45), (1025, 40, 9), (3001, 300, 64),
                                   (5000, 3, 130)])
def test_gradient(ctx, n, v, w, kind):
    check_gradient(ctx, n, v, w, kind)


@pytest.mark.parametrize("types", ["f32-f16", "bf16-f32", "bf16-bf16", "f16-f32", "f16-f16"])
@pytest.mark.parametrize("n,v,w,extra,lead", [(300, 50, 45, 14, 3), (70, 20, 1027, 0, 1), (513, 17, 8, 0, 0),
                                              (40, 30, 4096, 0, 0), (900, 64, 27, 2, 0)])
def test_gradient_types_and_strides(ctx, n, v, w, extra, lead, types):
    tn, on = types.split("-")
    check_gradient(ctx, n, v, w, "zipf", tn, on, "i64", extra, lead)
    check_gradient(ctx, n, v, w, "masked", tn, on, "i32", extra, lead, padding=2)


@pytest.mark.parametrize("n,v,w,kind", [(100_003, 2000, 12, "zipf"), (60_000, 3, 7, "hot"), (40_001, 70_000, 4, "uniform"),
                                        (33_000, 500, 100, "one"), (17_000, 900, 48, "masked"), (16_384, 64, 33, "zipf"),
                                        (16_385, 64, 33, "sorted"), (50_000, 1 << 20, 3, "distinct")])
def test_gradient_of_many_positions(ctx, n, v, w, kind):
    check_gradient(ctx, n, v, w, kind)
    check_gradient(ctx, n, v, w, kind, "bf16", "f32", "i64", extra=3, accumulate=True, padding=v // 2)


def test_gradient_accumulates(ctx):
    for on in ("f32", "bf16"):
        check_gradient(ctx, 700, 90, 45, "zipf", "f32", on, accumulate=True)
        check_gradient(ctx, 3, 2000, 64, "uniform", "f32", on, accumulate=True)


def test_gradient_of_nothing_and_of_broadcast_rows(ctx):
    torch = _t()
    d = torch.full((5, 7), 3.0, device="cuda")
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    B.gs_embed_bwd(ctx, empty, torch.empty((0, 7), device="cuda"), d)
    assert d.eq(0.0).all()
    d.fill_(3.0)
    B.gs_embed_bwd(ctx, empty, torch.empty((0, 7), device="cuda"), d, accumulate=True)
    assert d.eq(3.0).all()
    # one gradient row for every position
    idx = torch.tensor([1, 1, 3, 1], dtype=torch.int32, device="cuda")
    row = torch.arange(7, dtype=torch.float32, device="cuda")
    B.gs_embed_bwd(ctx, idx, row.expand(4, 7), d)
    assert torch.equal(d[1], 3 * row) and torch.equal(d[3], row) and d[0].eq(0.0).all() and d[2].eq(0.0).all()


def test_masked_rows_are_not_read(ctx):
    torch = _t()
    idx = torch.tensor([0, -1, 2, 5, 2], device="cuda")
    x = torch.ones((5, 6), device="cuda")
    x[1], x[3] = float("nan"), float("inf")
    x[0] = float("nan")
    d = torch.empty((5, 6), device="cuda")
    B.gs_embed_bwd(ctx, idx, x, d, padding=0)
    assert d[2].eq(2.0).all() and d[0].eq(0.0).all() and d[[1, 3, 4]].eq(0.0).all()


def test_gradient_is_that_of_the_lookup(ctx):
    """Differences of L(table) = <weight, lookup(table)> along random
    directions equal <gradient, direction>; values chosen so that every
    product and sum is exact."""
    torch = _t()
    g = torch.Generator().manual_seed(3)
    n, v, w = 400, 37, 21
    ints = lambda *s: torch.randint(-8, 9, s, generator=g).float().cuda()
    table, weight = ints(v, w), ints(n, w)
    idx = torch.from_numpy(sample_index(n, v, "masked", 4)).cuda()
    d = torch.empty((v, w), device="cuda")
    B.gs_embed_bwd(ctx, idx, weight, d, scale=0.5)
    for k in range(5):
        e = ints(v, w)
        hi, lo = B.gs_embed_fwd(ctx, table + e, idx, scale=0.5), B.gs_embed_fwd(ctx, table - e, idx, scale=0.5)
        diff = ((hi.double() - lo.double()) * weight.double()).sum() / 2
        assert float(diff) == float((d.double() * e.double()).sum())


# ---------------------------------------------------------------------------- norm and clip

def make_list(sizes, name, seed=0, scale=1.0, lead=0):
    """Tensors of the given sizes in one flat buffer, nothing between them."""
    torch = _t()
    g = torch.Generator().manual_seed(seed)
    flat = (torch.randn(lead + sum(sizes), generator=g) * scale).to(dtype(name)).cuda()
    at, out = lead, []
    for s in sizes:
        out.append(flat[at:at + s])
        at += s
    return out


LISTS = [[1], [0, 3, 0], [5, 1023, 1024, 1025, 2, 4097], [70_001], [1] * 300, list(range(1, 260, 7)) * 5, [300_007, 11]]


def reference_norm(ts):
    return math.sqrt(sum(float((f64(t) ** 2).sum()) for t in ts))


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", LISTS)
def test_norm_and_clip(ctx, sizes, name):
    torch = _t()
    ts = make_list(sizes, name, seed=len(sizes), lead=1)
    outs = make_list(sizes, name, seed=1, lead=2)
    norm = reference_norm(ts)
    U, tiny = UNIT[name]
    for limit in (0.5 * norm, 3.0 * norm + 1.0, 0.0, float("inf")):
        c = min(1.0, limit / (norm + 1e-6))
        r = B.gs_grad_norm(ctx, ts, limit)
        close(r[0], norm, 2 * u * norm)
        close(r[1], c, 2 * u * c)
        keep = [t.clone() for t in ts]
        r2 = B.gs_clip_grads(ctx, B.TensorList(ts), limit, out=B.TensorList(outs))
        assert torch.equal(r, r2)
        for t, k, o in zip(ts, keep, outs):
            assert torch.equal(t, k)
            close(o, f64(t) * c, (4 * u + U) * np.abs(f64(t) * c) + tiny)
    # in place: the same bits
    limit = 0.25 * norm
    B.gs_clip_grads(ctx, ts, limit, out=outs)
    B.gs_clip_grads(ctx, ts, limit)
    for t, o in zip(ts, outs):
        assert torch.equal(t, o)


def test_norm_of_strided_columns_and_mixed_types(ctx):
    torch = _t()
    rows = torch.randn((777, 59), generator=torch.Generator().manual_seed(2)).cuda()
    half = torch.randn((31, 33), generator=torch.Generator().manual_seed(3)).half().cuda()
    ts = [rows[:, 0:3], rows[:, 10:11], rows[:, 11:], half, half[:, 5:6].float()[:, 0], rows[3:4, 7:40]]
    norm = reference_norm(ts)
    r = B.gs_grad_norm(ctx, ts, 1.0)
    close(r[0], norm, 2 * u * norm)
    want = [f64(t) / (norm + 1e-6) for t in ts[:3]]
    other = rows.clone()
    B.gs_clip_grads(ctx, ts, 1.0, out=[other[:, 0:3], other[:, 10:11], other[:, 11:], half.clone(), ts[4].clone(),
                                       torch.empty_like(ts[5])])
    for o, w in zip([other[:, 0:3], other[:, 10:11], other[:, 11:]], want):
        close(o, w, 5 * u * np.abs(w))
    assert torch.equal(other[:, 3:10], rows[:, 3:10])
    # a broadcast row counts once for each of its rows
    row = torch.full((5,), 2.0, device="cuda")
    close(B.gs_grad_norm(ctx, [row.expand(9, 5)])[0], math.sqrt(180.0), 2 * u * math.sqrt(180.0))


def test_norm_of_extreme_values(ctx):
    torch = _t()
    inf, nan = float("inf"), float("nan")
    big = torch.full((1000,), 1e30, device="cuda")         # squares beyond f32
    close(B.gs_grad_norm(ctx, [big], 1.0)[0], float(big[0]) * math.sqrt(1000.0), 1e25)
    small = torch.full((1000,), 1e-30, device="cuda")      # squares below f32
    close(B.gs_grad_norm(ctx, [small], 1.0)[0], float(small[0]) * math.sqrt(1000.0), 1e-35)
    assert B.gs_grad_norm(ctx, [small], 1.0)[1] == 1.0
    x = torch.ones(5000, device="cuda")
    x[4999] = inf
    r = B.gs_grad_norm(ctx, [x], 1.0)
    assert r[0] == inf and r[1] == 0.0
    assert B.gs_grad_norm(ctx, [x])[0] == inf
    x[17] = nan
    assert B.gs_grad_norm(ctx, [x], 1.0).isnan().all()
    assert B.gs_grad_norm(ctx, []).tolist() == [0.0, 1.0]
    assert B.gs_grad_norm(ctx, [x[:0]], 1.0).tolist() == [0.0, 1.0]
    zero = torch.zeros(10, device="cuda")
    B.gs_clip_grads(ctx, [zero], 1.0)
    assert zero.eq(0.0).all()


# ---------------------------------------------------------------------------- Adam over lists

def adam_reference(p, m, v, g, c, o):
    x = g * c
    m1 = o["beta1"] * m + (1 - o["beta1"]) * x
    v1 = o["beta2"] * v + (1 - o["beta2"]) * x * x
    den = np.sqrt(v1 / (1 - o["beta2"] ** o["step"])) + o["eps"]
    upd = o["lr"] / (1 - o["beta1"] ** o["step"]) * m1 / den
    return p * (1 - o["lr"] * o["weight_decay"]) - upd, m1, v1, den, upd


def _adam_bounds(p, m, v, g, c, o, den, upd, v1):
    """The f32 evaluation's error: the scaled gradient 3u (the factor's 2u, a
    product); m: each term 2u more and the sum u; v: the square 7u, its factor
    and product 2u, the sum u; the root halves v's error; the update's
    quotient, product and constants 4u; the difference u of each term."""
    dm = 7 * u * (np.abs(o["beta1"] * m) + np.abs((1 - o["beta1"]) * g * c))
    dv = 12 * u * v1
    dp = 3 * u * (np.abs(p) + np.abs(upd)) + 12 * u * np.abs(upd) + \
        o["lr"] / (1 - o["beta1"] ** o["step"]) * dm / den
    return dp + 2.0 ** -140, dm + 2.0 ** -148, dv + 2.0 ** -148


def run_adam(ctx, params, grads, o, limit=None, copies=None, seed=0):
    torch = _t()
    gen = torch.Generator().manual_seed(seed)
    ms = [(torch.randn(p.shape, generator=gen) * 0.1).cuda() for p in params]
    vs = [((torch.randn(p.shape, generator=gen) * 0.1) ** 2).cuda() for p in params]
    old = [(f64(p), f64(m), f64(v), f64(g)) for p, m, v, g in zip(params, ms, vs, grads)]
    norm, c = None, 1.0
    if limit is not None:
        norm = B.gs_grad_norm(ctx, grads, limit)
        c = min(1.0, limit / (reference_norm(grads) + 1e-6))
    B.gs_adam_tensors(ctx, params, ms, vs, grads, norm=norm, copies=copies, **o)
    for k, (p, m, v, g) in enumerate(zip(params, ms, vs, grads)):
        p0, m0, v0, g0 = old[k]
        p1, m1, v1, den, upd = adam_reference(p0, m0, v0, g0.reshape(p0.shape), c, o)
        bp, bm, bv = _adam_bounds(p0, m0, v0, g0.reshape(p0.shape), c, o, den, upd, v1)
        close(p, p1, bp)
        close(m, m1, bm)
        close(v, v1, bv)
        if copies is not None and copies[k] is not None:
            assert torch.equal(copies[k], p.to(copies[k].dtype).reshape(copies[k].shape))


OPTS = dict(step=1, lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", LISTS)
def test_adam(ctx, sizes, name):
    grads = make_list(sizes, name, seed=4, lead=1)
    params = make_list(sizes, "f32", seed=5, lead=3)
    run_adam(ctx, params, grads, OPTS)
    run_adam(ctx, params, grads, dict(OPTS, step=1000, weight_decay=0.1, eps=1e-15), limit=0.5)
    run_adam(ctx, params, grads, dict(OPTS, step=3), limit=1e9, copies=make_list(sizes, "bf16", lead=1))


def test_adam_of_gradient_columns(ctx):
    torch = _t()
    gen = torch.Generator().manual_seed(6)
    rows = torch.randn((501, 59), generator=gen).cuda()
    params = [torch.randn(s, generator=gen).cuda() for s in ((501, 3), (501, 4), (501,), (501, 48), (7, 48))]
    table = torch.randn((7, 48), generator=gen).cuda()
    grads = [rows[:, 0:3], rows[:, 6:10], rows[:, 10:11], rows[:, 11:], table]
    params[2] = params[2].reshape(501, 1)
    copies = [None, torch.empty((501, 4), dtype=torch.float16, device="cuda"), None, None,
              torch.empty((7, 48), dtype=torch.bfloat16, device="cuda")]
    run_adam(ctx, params, grads, dict(OPTS, step=9), limit=2.0, copies=copies)


def test_adam_leaves_a_step_out_whose_norm_is_not_finite(ctx):
    torch = _t()
    for bad in (float("inf"), float("nan")):
        g = torch.ones(3000, device="cuda")
        g[2999] = bad
        p, m, v = (torch.full((3000,), x, device="cuda") for x in (1.0, 2.0, 3.0))
        low = torch.full((3000,), 4.0, dtype=torch.bfloat16, device="cuda")
        norm = B.gs_grad_norm(ctx, [g], 1.0)
        B.gs_adam_tensors(ctx, [p], [m], [v], [g], norm=norm, copies=[low], **OPTS)
        assert p.eq(1.0).all() and m.eq(2.0).all() and v.eq(3.0).all() and low.eq(4.0).all()


def test_adam_of_zero_gradients_moves_nothing(ctx):
    torch = _t()
    p = torch.randn(1000, device="cuda")
    old, z = p.clone(), torch.zeros(1000, device="cuda")
    m, v = z.clone(), z.clone()
    B.gs_adam_tensors(ctx, [p], [m], [v], [z], step=1, eps=1e-15)
    assert torch.equal(p, old) and m.eq(0).all() and v.eq(0).all()


def test_adam_agrees_with_the_scene_update(ctx):
    """gs_adam_tensors over a scene's five groups and gs_train_view's update
    from the same dense gradient: the same moments and parameters to the
    rounding of the two evaluations (hardware reciprocal and root there)."""
    torch = _t()
    from differentiable_gaussian_splatting_amd import scenes
    w = scenes.make_workload("c1_small", n=900, width=80, height=64, seed=21, sh_degree=3)
    target = torch.from_numpy(w.target).cuda()
    a, b = B.DeviceScene(w.scene), B.DeviceScene(w.scene)
    ma, va, mb, vb = (B.like_scene(a) for _ in range(4))
    g3 = torch.zeros((900, 59), device="cuda")
    B.gs_train_view(ctx, w.camera, a, target, grad3d_out=g3)
    B.gs_train_view(ctx, w.camera, a, target, adam=dict(step=1, params=a, m=ma, v=va, lr=1e-3, eps=1e-8))
    grads = [g3[:, 0:3], g3[:, 3:6], g3[:, 6:10], g3[:, 10], g3[:, 11:]]
    grads[3] = g3[:, 10:11]
    ps = [t.reshape(900, -1) for t in b.tensors()]
    B.gs_adam_tensors(ctx, ps, [t.reshape(900, -1) for t in mb.tensors()], [t.reshape(900, -1) for t in vb.tensors()],
                      grads, step=1, lr=1e-3, eps=1e-8)
    # the view's gradient sums its atomics in another order from run to run, and a first step is
    # lr sign(g) wherever |g| >> eps: where the gradient is not tiny both agree to that order's rounding
    g = torch.cat([x.reshape(-1) for x in grads])
    pa = torch.cat([t.reshape(-1) for t in a.tensors()])
    pb = torch.cat([t.reshape(-1) for t in ps])
    sure = g.abs() > 1e-6
    assert int(sure.sum()) > 1000
    assert float((pa - pb)[sure].abs().max()) <= 1e-5


# ---------------------------------------------------------------------------- streams, graphs, refusals

def test_context_on_another_stream(ctx):
    torch = _t()
    side = torch.cuda.Stream()
    c = B.Context(stream=side)
    table, idx = torch.randn((50, 33), device="cuda"), torch.randint(0, 50, (4000,), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    out = B.gs_embed_fwd(c, table, idx)
    d = torch.empty_like(table)
    side.wait_stream(torch.cuda.current_stream())
    B.gs_embed_bwd(c, idx, out, d)
    norm = B.gs_clip_grads(c, [d], 1.0)
    torch.cuda.current_stream().wait_stream(side)
    want = torch.empty_like(table)
    B.gs_embed_bwd(ctx, idx, B.gs_embed_fwd(ctx, table, idx), want)
    n2 = B.gs_clip_grads(ctx, [want], 1.0)
    assert torch.equal(d, want) and torch.equal(norm, n2)
    torch.cuda.synchronize()
    c.close()


def test_graph_replays(ctx):
    torch = _t()
    stream = torch.cuda.Stream()
    c = B.Context(stream=stream)
    n, v, w = 6000, 200, 24
    table, idx = torch.randn((v, w), device="cuda"), torch.randint(0, v, (n,), dtype=torch.int32, device="cuda")
    out, d, norm = torch.empty((n, w), device="cuda"), torch.empty((v, w), device="cuda"), torch.empty(2, device="cuda")
    p, m, s = table.clone(), torch.zeros_like(table), torch.zeros_like(table)

    def step(cc):
        B.gs_embed_fwd(cc, p, idx, out)
        B.gs_embed_bwd(cc, idx, out, d)
        B.gs_clip_grads(cc, [d], 1.0, norm)
        B.gs_adam_tensors(cc, [p], [m], [s], [d], step=5, norm=norm)

    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step(c)          # the first use allocates
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(c)
    for rep in range(4):
        for t, val in ((p, table), (m, torch.zeros_like(m)), (s, torch.zeros_like(s))):
            t.copy_(val * (1 + rep))
        idx.copy_(torch.randint(0, v, (n,), dtype=torch.int32, device="cuda"))
        keep = [t.clone() for t in (p, m, s)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, d, norm, p, m, s)]
        for t, k in zip((p, m, s), keep):
            t.copy_(k)
        step(ctx)
        torch.cuda.synchronize()
        for a, b in zip(got, (out, d, norm, p, m, s)):
            assert torch.equal(a, b), rep
    c.close()


def test_allocation_failure_leaves_outputs(ctx):
    torch = _t()
    from tests.test_gpu_errors import FailingContext
    f = FailingContext()
    idx, x = torch.randint(0, 70, (40_000,), device="cuda"), torch.randn((40_000, 5), device="cuda")
    d = torch.full((70, 5), 2.0, device="cuda")
    g = [torch.randn(5000, device="cuda")]
    norm = torch.full((2,), 9.0, device="cuda")
    large = [torch.randn(500_000, device="cuda")]
    norm2 = norm.clone()
    live = f.mem_stats()["live"]
    # a list as small as g is clipped without an allocation
    for call, same, allocates in ((lambda: B.gs_embed_bwd(f, idx, x, d), lambda: d.eq(2.0).all(), True),
                                  (lambda: B.gs_clip_grads(f, g, 1e-3, norm), lambda: norm.eq(9.0).all(), False),
                                  (lambda: B.gs_clip_grads(f, large, 1e-3, norm2),
                                   lambda: norm2.eq(9.0).all() and torch.equal(large[0], kept), True)):
        keep, kept = g[0].clone(), large[0].clone()
        k = 1
        while True:
            f.arm(k)
            try:
                call()
                break
            except B.GsError as e:
                assert e.status == B.GS_ERR_OOM
                torch.cuda.synchronize()
                assert same() and torch.equal(g[0], keep) and f.mem_stats()["live"] == live
            k += 1
        f.arm(0)
        assert (k > 1) == allocates and f.mem_stats()["live"] == live
    f.close()


def refused(status, fn):
    with pytest.raises(B.GsError) as e:
        fn()
    assert e.value.status == status, str(e.value)


def test_refusals(ctx):
    torch = _t()
    bad = B.GS_ERR_INVALID_ARG
    table, idx = torch.randn((4, 6), device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty((3, 6), device="cuda")
    refused(bad, lambda: B.gs_embed_fwd(ctx, table, idx, out[:2]))
    refused(bad, lambda: B.gs_embed_fwd(ctx, table, idx, out[:, :5]))
    refused(bad, lambda: B.gs_embed_fwd(ctx, table, idx, out[:1].expand(3, 6)))       # written rows overlap
    refused(bad, lambda: B.gs_embed_bwd(ctx, idx, out[:2], table))
    refused(bad, lambda: B.gs_embed_bwd(ctx, idx, out, table.as_strided((4, 6), (5, 1))))
    refused(bad, lambda: B.gs_grad_norm(ctx, [out], -1.0))
    refused(bad, lambda: B.gs_grad_norm(ctx, [out], float("nan")))
    refused(bad, lambda: B.gs_clip_grads(ctx, [out], 1.0, out=[out[:2]]))
    refused(bad, lambda: B.gs_clip_grads(ctx, [out], 1.0, out=[out.half()]))
    refused(bad, lambda: B.gs_clip_grads(ctx, [out[:1].expand(3, 6)], 1.0))
    p = [torch.randn(5, device="cuda") for _ in range(4)]
    adam = lambda **kw: B.gs_adam_tensors(ctx, [p[0]], [p[1]], [p[2]], [kw.pop("g", p[3])], **{**OPTS, **kw})
    for kw in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan")),
               dict(weight_decay=float("inf")), dict(g=torch.randn(4, device="cuda"))):
        refused(bad, lambda: adam(**kw))
    refused(bad, lambda: B.gs_adam_tensors(ctx, [p[0].half()], [p[1]], [p[2]], [p[3]], **OPTS))
    wide = torch.randn((5, 8), device="cuda")
    refused(bad, lambda: B.gs_adam_tensors(ctx, [wide[:, :4]], [wide[:, 4:]], [wide[:, 4:]], [wide[:, 4:]], **OPTS))
    with pytest.raises(ValueError):
        B.gs_embed_fwd(ctx, table.double(), idx)
    with pytest.raises(ValueError):
        B.gs_embed_fwd(ctx, table.t(), idx)
    with pytest.raises(ValueError):
        B.gs_embed_fwd(ctx, table, idx.float())
    with pytest.raises(ValueError):
        B.gs_embed_fwd(ctx, table.cpu(), idx)
    with pytest.raises(ValueError):
        B.gs_embed_fwd(ctx, table, torch.zeros((3, 2), dtype=torch.int32, device="cuda")[:, 0])
    with pytest.raises(ValueError):
        B.gs_grad_norm(ctx, [out], norm=torch.empty(1, device="cuda"))
    with pytest.raises(ValueError):
        B.gs_adam_tensors(ctx, [p[0]], [p[1]], [p[2]], [], **OPTS)


def test_refusals_at_the_c_entries(ctx):
    """Descriptors that the binding would not make."""
    torch = _t()
    L, h = ctx.lib, ctx.handle
    x = torch.randn((4, 6), device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    norm = torch.empty(2, device="cuda")
    T = lambda **kw: B.gs_tensor(*[{**dict(data=x.data_ptr(), rows=4, cols=6, stride=6, type=0, pad=0), **kw}[k]
                                   for k in ("data", "rows", "cols", "stride", "type", "pad")])
    bad, over = B.GS_ERR_INVALID_ARG, B.GS_ERR_OVERFLOW
    ok = T()
    for t, st in ((T(type=3), bad), (T(type=-1), bad), (T(rows=-1), bad), (T(cols=-1), bad), (T(stride=-6), bad),
                  (T(data=0), bad), (T(data=x.data_ptr() + 1), bad), (T(rows=1 << 41, stride=0), over),
                  (T(rows=1 << 31, cols=1, stride=0), over)):
        assert L.gs_embed_fwd(h, C.byref(t), i.data_ptr(), B.GS_I32, 4, 1.0, C.byref(ok)) == st
        assert B.gs_grad_norm and L.gs_last_error(h)
    assert L.gs_embed_fwd(h, None, i.data_ptr(), B.GS_I32, 4, 1.0, C.byref(ok)) == bad
    assert L.gs_embed_fwd(h, C.byref(ok), None, B.GS_I32, 4, 1.0, C.byref(ok)) == bad
    assert L.gs_embed_fwd(h, C.byref(ok), i.data_ptr() + 2, B.GS_I32, 4, 1.0, C.byref(ok)) == bad
    assert L.gs_embed_fwd(h, C.byref(ok), i.data_ptr(), B.GS_F32, 4, 1.0, C.byref(ok)) == bad
    assert L.gs_embed_fwd(h, C.byref(ok), i.data_ptr(), B.GS_I32, -1, 1.0, C.byref(ok)) == bad
    assert L.gs_embed_bwd(h, i.data_ptr(), B.GS_I32, 1 << 31, C.byref(ok), 1.0, -1, 0, C.byref(ok)) == over
    assert L.gs_embed_fwd(None, C.byref(ok), i.data_ptr(), B.GS_I32, 4, 1.0, C.byref(ok)) == bad
    assert L.gs_grad_norm(h, None, 1, 1.0, norm.data_ptr()) == bad
    assert L.gs_grad_norm(h, C.cast(C.pointer(ok), C.c_void_p), 1, 1.0, None) == bad
    assert L.gs_grad_norm(h, C.cast(C.pointer(ok), C.c_void_p), -1, 1.0, norm.data_ptr()) == bad
    q = C.cast(C.pointer(ok), C.c_void_p)
    assert L.gs_adam_tensors(h, q, q, q, q, None, 1, None, None) == bad
    assert L.gs_adam_tensors(h, None, q, q, q, None, 1, C.byref(B.gs_adam_opts(1, 0, 1e-3, 0.9, 0.999, 1e-8, 0.0)),
                             None) == bad


@pytest.mark.parametrize("n", [65_536, 65_537, 70_001])
@pytest.mark.parametrize("v,kind", [(1, "uniform"), (2, "masked"), (511, "zipf"), (512, "sorted"), (513, "uniform"),
                                    (300_000, "masked"), ((1 << 20) + 3, "uniform"), (40, "none"), (1, "masked")])
def test_gradient_around_the_sorts_limits(ctx, n, v, kind):
    """Both ways of grouping, one to three passes, and rows at the bits' edges."""
    check_gradient(ctx, n, v, 2, kind, index="i64" if v % 2 else "i32")


@pytest.mark.parametrize("w", [1, 2, 3, 4, 5, 7, 8, 255, 256, 257, 258, 511, 512, 513, 1025])
def test_gradient_widths(ctx, w):
    """Widths around the packs and column ranges, each accumulated too (columns that two lanes hold are added once)."""
    for tn in ("f32", "bf16"):
        check_gradient(ctx, 300, 11, w, "zipf", tn, "f32")
        check_gradient(ctx, 300, 11, w, "hot", tn, "f32", accumulate=True)


@pytest.mark.parametrize("count", [61, 62, 63, 107, 108, 109, 143, 144, 145, 200])
def test_lists_around_a_launchs_tensors(ctx, count):
    """Lists around the tensors of one launch, small and (with one large tensor) described in a table."""
    torch = _t()
    for big in (0, 4_100_000):
        sizes = [k % 7 for k in range(count)] + ([big] if big else [])
        ts, outs = make_list(sizes, "f32", seed=count), make_list(sizes, "f32", seed=1, lead=1)
        norm = reference_norm(ts)
        r = B.gs_clip_grads(ctx, ts, 0.5 * norm, out=outs)
        close(r[0], norm, 2 * u * norm)
        c = 0.5 * norm / (norm + 1e-6)
        for t, o in zip(ts, outs):
            close(o, f64(t) * c, 5 * u * np.abs(f64(t) * c) + 2.0 ** -149)
        run_adam(ctx, outs, ts, OPTS, limit=0.1, copies=make_list(sizes, "f16", lead=3))


def test_lists_of_many_column_views(ctx):
    """More tensors with rows apart than a launch holds, in a small list and in one large enough for a table."""
    torch = _t()
    gen = torch.Generator().manual_seed(8)
    for rows in (9, 60_000):
        wide = torch.randn((rows, 150), generator=gen).cuda()
        grads = [wide[:, 2 * k:2 * k + 1] for k in range(70)]
        norm = reference_norm(grads)
        close(B.gs_grad_norm(ctx, grads, 1.0)[0], norm, 2 * u * norm)
        params = [torch.randn((rows, 1), generator=gen).cuda() for _ in grads]
        run_adam(ctx, params, grads, OPTS, limit=1.0)
        out = wide.clone()
        B.gs_clip_grads(ctx, grads, 0.5 * norm, out=[out[:, 2 * k:2 * k + 1] for k in range(70)])
        c = 0.5 * norm / (norm + 1e-6)
        close(out[:, 0:140:2], f64(wide[:, 0:140:2]) * c, 5 * u * np.abs(f64(wide[:, 0:140:2]) * c))
        assert torch.equal(out[:, 1:140:2], wide[:, 1:140:2])


@pytest.mark.parametrize("n", [8, 9, 64, 127, 128, 129, 255, 256, 257, 511, 512, 513])
@pytest.mark.parametrize("w", [1, 3, 48, 257, 300])
def test_gradient_of_few_positions(ctx, n, w):
    """Around the sizes that one block sums, with rows to clear beside them."""
    for kind in ("one", "zipf", "masked"):
        check_gradient(ctx, n, 700, w, kind, "bf16" if n % 2 else "f32", "f32", "i64" if w == 3 else "i32", padding=5)
    check_gradient(ctx, n, 70, w, "uniform", "f32", "bf16", accumulate=True)


# ---------------------------------------------------------------------------- lists at the limits of a launch

def long_list(kind):
    """(tensors, buffer) of lists of more than four million values whose descriptors go to a table on the device:
    columns of wide rows, or dense tensors."""
    torch = _t()
    gen = torch.Generator().manual_seed(11)
    if kind == "columns":
        wide = torch.randn((70_001, 130), generator=gen).cuda()
        return [wide[:, 2 * k:2 * k + 1] for k in range(65)], wide
    ts = make_list([11] * 432 + [4_200_000], "f32", seed=12)
    return ts, ts[0]._base


@pytest.mark.parametrize("kind", ["columns", "dense"])
def test_allocation_failure_leaves_the_outputs_of_a_long_list(kind):
    """Every allocation of a call fails in turn, the descriptor tables among them: norm, outputs, parameters and
    moments keep their values."""
    torch = _t()
    from tests.test_gpu_errors import FailingContext
    f = FailingContext()
    ts, buf = long_list(kind)
    norm = torch.full((2,), 9.0, device="cuda")
    outs = [torch.full_like(t, 5.0) for t in ts]
    p, m, v = ([torch.full(t.shape, x, device="cuda") for t in ts] for x in (1.0, 2.0, 3.0))
    lists = [B.TensorList(x) for x in (ts, outs, p, m, v)]
    keep = buf.clone()
    full = lambda xs, x: all(bool(t.eq(x).all()) for t in xs)
    untouched = lambda: (bool(norm.eq(9.0).all()) and torch.equal(buf, keep) and full(outs, 5.0) and full(p, 1.0) and
                         full(m, 2.0) and full(v, 3.0))
    live = f.mem_stats()["live"]
    for call in (lambda: B.gs_grad_norm(f, lists[0], 1e-3, norm), lambda: B.gs_clip_grads(f, lists[0], 1e-3, norm),
                 lambda: B.gs_clip_grads(f, lists[0], 1e-3, norm, out=lists[1]),
                 lambda: B.gs_adam_tensors(f, *lists[2:], lists[0], **OPTS)):
        k = 1
        while True:
            f.arm(k)
            try:
                call()
                break
            except B.GsError as e:
                assert e.status == B.GS_ERR_OOM
                torch.cuda.synchronize()
                assert untouched(), k
                assert f.mem_stats()["live"] == live
            k += 1
        f.arm(0)
        assert k > 2
        buf.copy_(keep)
        norm.fill_(9.0)
        for t in outs:
            t.fill_(5.0)
    f.close()


def test_adam_of_tensors_without_values(ctx):
    """Rows without columns and columns without rows take part in a list and change nothing in it."""
    torch = _t()
    gen = torch.Generator().manual_seed(14)
    shapes = [(5, 0), (7, 3), (0, 4), (1, 0), (0,), (6,)]
    params, grads = ([torch.randn(s, generator=gen).cuda() for s in shapes] for _ in range(2))
    assert params[0].stride() == (1, 1)
    run_adam(ctx, params, grads, OPTS, copies=[torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes])
    r = B.gs_grad_norm(ctx, grads, 1.0)
    norm = reference_norm(grads)
    close(r[0], norm, 2 * u * norm)


@pytest.mark.parametrize("n", [2, 200, 1500])
def test_gradient_of_very_wide_rows(ctx, n):
    """More column ranges than a launch has blocks in y: 2 positions (one launch), 200 (one block of positions per
    range), and 1500 that share one gradient row (several, joined).  Whole numbers, so that every sum is exact."""
    torch = _t()
    w = 256 * 65_536 + 5
    row = (torch.arange(w, device="cuda") % 5 - 2).float()
    dout = row.expand(n, w) if n > 2 else torch.stack([row, -3.0 * row])
    idx = torch.full((n,), 2, dtype=torch.int32, device="cuda")
    idx[1] = 0
    d = torch.full((3, w), 7.0, device="cuda")
    B.gs_embed_bwd(ctx, idx, dout, d, scale=0.5)
    assert torch.equal(d[0], 0.5 * dout[1]) and d[1].eq(0.0).all() and torch.equal(d[2], 0.5 * (n - 1) * row)
    B.gs_embed_bwd(ctx, idx, dout, d, scale=0.5, accumulate=True)
    assert torch.equal(d[0], dout[1]) and d[1].eq(0.0).all() and torch.equal(d[2], (n - 1) * row)


def test_rows_in_the_shape_of_their_indices(ctx):
    """Indices (B, T) and contiguous rows (B, T, W), as a model holds them."""
    torch = _t()
    gen = torch.Generator().manual_seed(15)
    table, idx = torch.randn((9, 12), generator=gen).cuda(), torch.randint(-1, 9, (3, 5), generator=gen).cuda()
    out = torch.empty((3, 5, 12), device="cuda")
    assert B.gs_embed_fwd(ctx, table, idx, out) is out
    assert torch.equal(out.view(15, 12), B.gs_embed_fwd(ctx, table, idx))
    d, want = torch.empty_like(table), torch.empty_like(table)
    B.gs_embed_bwd(ctx, idx, out, d)
    B.gs_embed_bwd(ctx, idx, out.view(15, 12), want)
    assert torch.equal(d, want)
    one = torch.empty((1, 12), device="cuda")
    assert torch.equal(B.gs_embed_fwd(ctx, table, idx[0, 1], one[0])[None], B.gs_embed_fwd(ctx, table, idx[0, 1:2]))
    # rows that are not those of the indices
    for bad in (torch.empty((3, 5, 11), device="cuda"), torch.empty((5, 3, 24), device="cuda"),
                torch.empty((3, 4, 12), device="cuda")):
        with pytest.raises((ValueError, B.GsError)):
            B.gs_embed_bwd(ctx, idx, bad, d)
        with pytest.raises((ValueError, B.GsError)):
            B.gs_embed_fwd(ctx, table, idx, bad)
    with pytest.raises(ValueError):
        B.gs_embed_bwd(ctx, idx, out.transpose(0, 1), d)


@pytest.mark.parametrize("count", [3000, 3072, 3073, 5000])
def test_norm_and_clip_of_many_small_tensors(ctx, count):
    """Around the number of partials above which the factor has a launch of its own."""
    torch = _t()
    ts = make_list([40] * count, "f32", seed=21, lead=1)
    flat = ts[0]._base[1:]
    norm = float((f64(flat) ** 2).sum()) ** 0.5
    for limit in (0.25 * norm, 2.0 * norm + 1.0):
        c = min(1.0, limit / (norm + 1e-6))
        outs = make_list([40] * count, "f32", seed=1)
        r = B.gs_clip_grads(ctx, ts, limit, out=outs)
        close(r[0], norm, 2 * u * norm)
        close(r[1], c, 2 * u * c)
        close(outs[0]._base, f64(flat) * c, 5 * u * np.abs(f64(flat) * c))
        keep = outs[0]._base.clone()
        before = flat.clone()
        assert torch.equal(B.gs_clip_grads(ctx, ts, limit), r) and torch.equal(flat, keep)
        flat.copy_(before)


def test_clip_of_many_small_tensors_takes_time_in_proportion(ctx):
    """100,000 tensors of 40 values: norm and scaling together take a few times the norm's time (2.3 measured; 12
    when every block of the scaling adds the partials of all tensors)."""
    import time
    torch = _t()
    ts = B.TensorList(make_list([40] * 100_000, "f32", seed=22))
    norm = torch.empty(2, device="cuda")

    def seconds(call):
        call()
        times = []
        for _ in range(3):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            times.append(time.perf_counter() - t0)
        return min(times)

    alone = seconds(lambda: B.gs_grad_norm(ctx, ts, 1.0, norm))
    both = seconds(lambda: B.gs_clip_grads(ctx, ts, 1.0, norm))
    assert both < 6.0 * alone, (both, alone)


def mixed_list(live, big, seed):
    """`live` tensors with values, every ninth of them a column of wide rows, an empty one after every fifth, and
    the last one of `big` values where big > 0; beside them contiguous tensors of the same shapes."""
    torch = _t()
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((13, 2 * (live // 9) + 2), generator=g).cuda()
    ts, column = [], 0
    for k in range(live):
        if k % 9 == 4:
            ts.append(wide[:, 2 * column:2 * column + 1])
            column += 1
        else:
            ts.append(torch.randn(big if big and k == live - 1 else 1 + k % 6, generator=g).cuda())
        if k % 5 == 2:
            ts.append(torch.empty(0, device="cuda"))
    return ts, [torch.randn(t.shape, generator=g).cuda() for t in ts]


# tensors that one launch describes in its arguments: Adam 62, clip 108, norm 144; a list of more than four million
# values has them in a table from three times as many on
LIMITS = [61, 62, 63, 107, 108, 109, 143, 144, 145, 185, 186, 187, 323, 324, 325, 431, 432, 433, 500]


@pytest.mark.parametrize("big", [0, 4_100_000])
@pytest.mark.parametrize("live", LIMITS)
def test_lists_at_the_limits_of_a_launch(ctx, live, big):
    torch = _t()
    ts, outs = mixed_list(live, big, live)
    assert sum(t.numel() > 0 for t in ts) == live
    whole = np.concatenate([f64(t).ravel() for t in ts])
    norm = math.sqrt(float((whole ** 2).sum()))
    c = min(1.0, 0.5 * norm / (norm + 1e-6))
    r = B.gs_grad_norm(ctx, ts, 0.5 * norm)
    close(r[0], norm, 2 * u * norm)
    close(r[1], c, 2 * u * c)
    assert torch.equal(B.gs_clip_grads(ctx, ts, 0.5 * norm, out=outs), r)
    got = np.concatenate([f64(o).ravel() for o in outs])
    assert (np.abs(got - whole * c) <= 5 * u * np.abs(whole * c)).all()
    gen = torch.Generator().manual_seed(live)
    ps, ms = ([torch.randn(t.shape, generator=gen).cuda() for t in ts] for _ in range(2))
    vs = [torch.rand(t.shape, generator=gen).cuda() for t in ts]
    low = [torch.empty(t.shape, dtype=torch.float16, device="cuda") if k % 4 else None for k, t in enumerate(ts)]
    flat = lambda xs: np.concatenate([f64(x).ravel() for x in xs])
    old = [flat(x) for x in (ps, ms, vs)]
    o = dict(OPTS, step=3)
    B.gs_adam_tensors(ctx, ps, ms, vs, ts, norm=r, copies=low, **o)
    p1, m1, v1, den, upd = adam_reference(*old, whole, c, o)
    for x, want, bound in zip((ps, ms, vs), (p1, m1, v1), _adam_bounds(*old, whole, c, o, den, upd, v1)):
        assert (np.abs(flat(x) - want) <= bound).all()
    for p, k in zip(ps, low):
        assert k is None or torch.equal(k, p.half())
    B.gs_clip_grads(ctx, ts, 0.5 * norm)
    for t, x in zip(ts, outs):
        assert torch.equal(t, x)


@pytest.mark.parametrize("v,on", [((1 << 27) + 5, "f32"), ((1 << 31) - 1, "bf16")])
def test_gradient_of_more_rows_than_three_passes_sort(ctx, v, on):
    """Rows of 28 and 31 bits, grouped in four passes.  Whole numbers: every sum is exact."""
    torch = _t()
    n = 70_001
    rng = np.random.default_rng(31)
    # rows that differ in every digit, the first and last among them, and positions that name none
    names = np.unique(np.concatenate([[0, 1, v - 2, v - 1], rng.integers(0, v, 3000), 1 << np.arange(27)]))
    i = np.where(rng.random(n) < 0.1, rng.choice([-1, v, v + 1], n), rng.choice(names, n))
    x = rng.integers(-3, 4, n)
    d = torch.full((v, 1), 5.0, dtype=dtype(on), device="cuda")
    B.gs_embed_bwd(ctx, torch.from_numpy(i).cuda(), torch.from_numpy(x).float()[:, None].cuda(), d)
    sums = np.zeros(names.size)
    inside = (i >= 0) & (i < v)
    np.add.at(sums, np.searchsorted(names, i[inside]), x[inside].astype(np.float64))
    at = torch.from_numpy(names).cuda()
    got = d[at, 0]
    assert torch.equal(got, torch.from_numpy(sums).float().to(dtype(on)).cuda())
    d[at] = 0.0
    assert not any(bool(part.any()) for part in d.split(1 << 28))


def test_sizes_beyond_the_limits_are_refused(ctx):
    """OVERFLOW from each entry, by descriptors of broadcast rows (nothing is launched)."""
    torch = _t()
    L, h, over = ctx.lib, ctx.handle, B.GS_ERR_OVERFLOW
    x, norm = torch.zeros(64, device="cuda"), torch.empty(2, device="cuda")
    idx = torch.zeros(4, dtype=torch.int32, device="cuda")
    T = lambda rows, cols, stride: B.gs_tensor(x.data_ptr(), rows, cols, stride, 0, 0)
    ref = C.byref
    huge, apart = T(1 << 31, 1 << 10, 0), T(2, 1 << 31, 0)
    for t in (huge, apart):
        assert L.gs_embed_fwd(h, ref(t), idx.data_ptr(), B.GS_I32, 4, 1.0, ref(T(4, t.cols, t.cols))) == over
        assert L.gs_embed_bwd(h, idx.data_ptr(), B.GS_I32, t.rows, ref(t), 1.0, -1, 0, ref(T(1, t.cols, t.cols))) == over
        a = C.cast((B.gs_tensor * 1)(t), C.c_void_p)
        o = B.gs_adam_opts(1, 0, 1e-3, 0.9, 0.999, 1e-8, 0.0)
        p = C.cast((B.gs_tensor * 1)(T(1, 8, 8)), C.c_void_p)
        assert L.gs_grad_norm(h, a, 1, 1.0, norm.data_ptr()) == over
        assert L.gs_clip_grads(h, a, 1, 1.0, a, norm.data_ptr()) == over
        assert L.gs_adam_tensors(h, p, p, p, a, None, 1, o, None) == over
    for n, rows, cols in ((1 << 31, 4, 8), (4, 1 << 31, 8), (4, 4, 1 << 31)):
        assert L.gs_embed_fwd(h, ref(T(rows, cols, 0 if cols < 99 else cols)), idx.data_ptr(), B.GS_I32, n, 1.0,
                              ref(T(4, 8, 8))) == over
    many = (B.gs_tensor * 5)(*[T(1 << 30, 1 << 10, 0) for _ in range(5)])   # 5 x 2^40 values
    assert L.gs_grad_norm(h, C.cast(many, C.c_void_p), 5, 1.0, norm.data_ptr()) == over
