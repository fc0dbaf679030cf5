"""How the layers' products are cut into tiles: csrc/layer_plan.h, compiled for the CPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tests.layer_calls import CALLS, NARROW

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_gaussian_splatting_amd",
                    "csrc")
SOURCE = """
#include "layer_plan.h"
extern "C" void plan(int units, int f32, int direct, const int64_t* s, int64_t* out)
{
    const gsm::TilePlan p = gsm::plan_tiles(units, f32, direct, gsm::ProductShape{s[0], s[1], s[2], s[3] != 0, s[4] != 0, s[5] != 0});
    const int64_t all[8] = {p.tile, p.tm, p.tn, p.full, p.splits, p.kper, p.floats, 0};
    for (int i = 0; i < 8; ++i) out[i] = all[i];
}
"""
TILES = {"f32": [(256, 128, 32), (128, 128, 32), (64, 64, 32), (64, 64, 32)],
         "odd": [(256, 256, 64), (128, 128, 64), (64, 64, 64), (64, 64, 64)]}
TILES["aligned"] = TILES["odd"]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    lib = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o", lib], check=True)
    lib = ctypes.CDLL(lib)

    def call(kind, mode, m, n, k, units=256):
        shape = (ctypes.c_int64 * 6)(m, n, k, mode == "dw", mode in ("dw", "dx"), mode == "gated")
        out = (ctypes.c_int64 * 8)()
        lib.plan(units, kind == "f32", kind == "aligned", shape, out)
        return list(out)[:7]
    return call


def products(call, n, k, f):
    """Rows, columns and inner length of a call's products."""
    return [("dx", n, k, f), ("dw", f, k, n)] if call == "bwd" else [(call, n, f, k)]


def way(tm, tn, full):
    return "whole" if full == tm * tn else "split" if full == 0 else "mixed"


def test_the_calls_reach_every_tile(plan):
    reached = set()
    for call, kind, n, k, f in CALLS:
        assert n > 64 and min(k, f) >= 128   # neither few rows nor narrow ones
        assert kind == "f32" or (k % 8 == 0 and f % 8 == 0 if kind == "aligned" else k % 2 and f % 2)
        for mode, a, b, c in products(call, n, k, f):
            tile, tm, tn, full, _, _, _ = plan(kind, mode, a, b, c)
            reached.add((kind, mode, tile, way(tm, tn, full)))
    want = {(kind, mode, tile, w) for kind in ("f32", "odd", "aligned") for mode in ("fwd", "gated", "dx", "dw")
            for tile in range(3) for w in ("whole", "mixed", "split")}
    # five tiles of 64 x 64 a unit: a last round of them is never worth a split of its own in 16 bits
    want -= {(kind, mode, 2, "mixed") for kind in ("odd", "aligned") for mode in ("fwd", "gated", "dx", "dw")}
    assert reached == want
    tiny = {mode for call, n, k, f in NARROW for mode, a, b, c in products(call, n, k, f) for kind in ("f32", "odd")
            if plan(kind, mode, a, b, c)[0] == 3}
    assert tiny == {"fwd", "gated", "dx", "dw"}


@pytest.mark.parametrize("units", [256, 64, 1])
def test_plans_cover_their_products(plan, units):
    """Tiles cover the results and splits k, none of them empty; the workspace holds the split tiles' sums."""
    sizes = [1, 7, 8, 63, 64, 65, 129, 500, 2049, 8192, 70000]
    for kind in ("f32", "odd", "aligned"):
        for mode in ("fwd", "gated", "dx", "dw"):
            for m in sizes:
                for n in sizes:
                    for k in [0] + sizes:
                        tile, tm, tn, full, splits, kper, floats = plan(kind, mode, m, n, k, units)
                        bm, bn, bk = TILES[kind][tile]
                        cols = n * (2 if mode == "gated" else 1)
                        assert (tm - 1) * bm < m <= tm * bm and (tn - 1) * bn < cols <= tn * bn
                        assert splits >= 1 and kper % bk == 0 and splits * kper >= k
                        assert k == 0 or (splits - 1) * kper < k
                        assert 0 <= full <= tm * tn and (splits > 1) == (full < tm * tn)
                        assert floats == (splits * (tm * tn - full) * bm * bn if splits > 1 else 0)
