"""The Muon update on every tile of its products and at the ends of f32's range, against 64 bits.  The bound is that of
muon_reference: 1e-6 of |X| after one step, 3e-4 after five, less than one wrong value or one dropped part makes."""
import math

import pytest

from differentiable_gaussian_splatting_amd import binding as B
from tests import muon_reference as M
from tests.muon_lists import LISTS
from tests.test_gpu_layers import _t, check_muon, ctx, u  # noqa: F401
from tests.test_gpu_tensors import dtype

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [0, 1])
def test_norms_beyond_the_largest_float(ctx, steps):
    """|u| of 3e39 to 6e40, whose inverse is no normal float; a large lr, so that the update outweighs the parameters."""
    check_muon(ctx, [(60, 40), (300, 200), (1100, 900)], scale=3e37, steps=steps, lr=1e4, decay=0.0)


def check(ctx, shapes, steps, name, nesterov=True, copy=None, seed=0, gap=0):
    """p starts at 0 with rate -1, so that it becomes X."""
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R = lambda r, c: torch.randn((r, c), generator=gen, device="cuda") * 0.01
    p = [torch.zeros(s, device="cuda") for s in shapes]
    m = [R(r, c) for r, c in shapes]
    g = [R(r, c + gap).to(dtype(name))[:, :c] for r, c in shapes]
    q = None if copy is None else [torch.full(s, float("nan"), dtype=dtype(copy), device="cuda") for s in shapes]
    old = [t.double() for t in m]
    B.gs_muon_tensors(ctx, p, m, g, lr=-1.0, momentum=0.95, nesterov=nesterov, steps=steps, copies=q)
    mu = float(torch.tensor(0.95, dtype=torch.float32))
    for k, (r, c) in enumerate(shapes):
        G = g[k].double()
        M1 = mu * old[k] + G
        U = G + mu * M1 if nesterov else M1
        off = 4 * u * float((G.abs() + old[k].abs()).norm()) / float(U.norm())   # two products and sums, each u of it
        X, e = M.newton_schulz(U, steps, off)
        rate = math.sqrt(max(1.0, r / c))
        err = float((p[k].double() / rate - X).norm())
        assert err <= e + 3 * u * float(X.norm()), (k, r, c, err, e, float(X.norm()))
        if q is not None:
            assert torch.equal(q[k], p[k].to(q[k].dtype))


@pytest.mark.parametrize("index", range(len(LISTS)), ids=lambda i: "{1}x{0[0]}-{0[1]}".format(LISTS[i][0], len(LISTS[i])))
def test_every_tile(ctx, index):
    check(ctx, LISTS[index], 1, "f32", seed=index)
    check(ctx, LISTS[index], 5, ("f32", "f16", "bf16")[index % 3], nesterov=index % 2 == 0, copy=("bf16", "f16")[index % 2],
          seed=index, gap=index % 4)


def test_matrices_of_one_block(ctx):
    shapes = [(64, 48), (48, 64), (128, 128), (1, 1), (1, 512), (512, 1), (33, 31), (20, 300), (300, 20), (128, 97), (7, 5)]
    check(ctx, shapes, 1, "f32")
    check(ctx, shapes, 5, "bf16", copy="f16", gap=3)
