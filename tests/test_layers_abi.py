"""Layout of the Muon options and the layer binding's own checks (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from differentiable_gaussian_splatting_amd import binding


def test_muon_options_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    st = binding.gs_muon_opts
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gs.h"', "int main(void) {",
             '    printf("%d %d %d %d %d\\n", GS_ACT_NONE, GS_ACT_RELU, GS_ACT_SILU, GS_ACT_GELU, GS_ACT_SIGMOID);',
             '    printf("%zu", sizeof(gs_muon_opts));']
    lines += [f'    printf(" %zu", offsetof(gs_muon_opts, {f[0]}));' for f in st._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["    return 0;", "}"]) + "\n")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-I", inc, str(src), "-o", str(tmp_path / "layout")], check=True)
    acts, layout = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split("\n")
    assert [int(v) for v in acts.split()] == list(binding.GS_ACTIVATIONS.values())
    assert [int(v) for v in layout.split()] == [ctypes.sizeof(st)] + [getattr(st, f[0]).offset for f in st._fields_]


def test_unknown_activations_are_refused():
    with pytest.raises(ValueError):
        binding._activation("tanh")
