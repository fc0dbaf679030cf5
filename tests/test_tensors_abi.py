"""Layout of the tensor-list structures and the binding's own checks (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from differentiable_gaussian_splatting_amd import binding


def test_structs_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = [binding.gs_tensor, binding.gs_adam_opts]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gs.h"', "int main(void) {",
             '    printf("types %d %d %d %d %d\\n", GS_F32, GS_F16, GS_BF16, GS_I32, GS_I64);']
    for st in structs:
        lines.append(f'    printf("{st.__name__} %zu", sizeof({st.__name__}));')
        lines += [f'    printf(" %zu", offsetof({st.__name__}, {f[0]}));' for f in st._fields_]
        lines.append('    printf("\\n");')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["    return 0;", "}"]) + "\n")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-I", inc, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = dict((line.split()[0], [int(x) for x in line.split()[1:]]) for line in
               subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.splitlines())
    assert got["types"] == [binding.GS_F32, binding.GS_F16, binding.GS_BF16, binding.GS_I32, binding.GS_I64]
    for st in structs:
        assert got[st.__name__] == [ctypes.sizeof(st)] + [getattr(st, f[0]).offset for f in st._fields_]


def test_host_tensors_are_refused():
    import torch
    with pytest.raises(ValueError):
        binding.tensor_struct(torch.zeros(3))
    with pytest.raises(ValueError):
        binding.TensorList([torch.zeros(3)])
    assert len(binding.TensorList([])) == 0
