"""How the Muon update cuts its products (csrc/muon_plan.h, compiled for the CPU), and what its tests' bound rejects."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tests import muon_reference as M
from tests.muon_lists import LISTS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_gaussian_splatting_amd",
                    "csrc")
SOURCE = """
#include "muon_plan.h"
struct Group { int32_t count; struct { int32_t rows, cols; } t[48]; };
extern "C" void plan(int units, int n, const int32_t* sides, int32_t* out)
{
    Group g;
    g.count = n;
    for (int k = 0; k < n; ++k) g.t[k] = {sides[2 * k], sides[2 * k + 1]};
    double us;
    int splits = 0;
    gsm::choose_sizes(units, g, &out[0], &splits);
    out[1] = splits;
    out[2] = gsm::choose_tile<gsm::kGram>(units, g, out[0], splits, &us);
    out[3] = gsm::choose_tile<gsm::kPoly>(units, g, out[0], 1, &us);
    out[4] = gsm::choose_tile<gsm::kNext>(units, g, out[0], 1, &us);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    lib = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o", lib], check=True)
    lib = ctypes.CDLL(lib)

    def call(shapes, units=256):
        sides = (ctypes.c_int32 * (2 * len(shapes)))(*[v for s in shapes for v in s])
        out = (ctypes.c_int32 * 5)()
        lib.plan(units, len(shapes), sides, out)
        return list(out)
    return call


def test_the_lists_reach_every_tile(plan):
    reached = set()
    for shapes in LISTS:
        tall = shapes[0][0] > shapes[0][1]
        assert all((r > c) == tall for r, c in shapes) and len(shapes) <= 48
        assert all(max(r, c) > 512 or min(r, c) > 128 for r, c in shapes)   # none fits one block
        unit, splits, gram, poly, nxt = plan(shapes)
        assert all(unit % M_TILE[t] == 0 for t in (gram, poly, nxt))
        reached |= {(tall, "G", gram, splits > 1), (tall, "P", poly), (tall, "X", nxt), (tall, unit)}
    for tall in (False, True):
        want = {(tall, "G", t, s) for t in range(3) for s in (False, True)} | {(tall, p, t) for p in "PX" for t in range(3)}
        want |= {(tall, n) for n in (64, 128, 256)}
        assert {r for r in reached if r[0] == tall} == want


M_TILE = (256, 128, 64)


@pytest.mark.parametrize("shape", [(131, 135), (257, 260), (64, 1200), (1047, 400), (300, 3), (1, 400)])
def test_the_bound_accepts_two_parts_and_nothing_less(shape):
    """An emulation of the steps with two f16 parts a factor stays well inside the bound; with one f16 or one bf16 part,
    with one tile of X lost, or with one value of X taken from its neighbour, it does not."""
    import torch
    v = torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))) * 0.01

    def tile(x):
        x[:64, :64] = 0

    def value(x):
        x[-1, -1] = x[0, 0]

    for steps in (1, 5):
        X, e = M.newton_schulz(v.double(), steps)
        err = lambda *a, **kw: float((M.emulated(v, steps, *a, **kw).double() - X).norm())
        assert err() <= 0.2 * e
        assert err(1) > e and err(1, torch.bfloat16) > 2 * e and err(spoil=tile) > 10 * e and err(spoil=value) > e
        assert e <= 3e-4 * float(X.norm())
