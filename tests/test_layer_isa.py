"""Checks on the gfx950 assembly of the layer operators' kernels (CPU only: hipcc cross-compiles): no
packed fp32 arithmetic, no spills in the memory-bound kernels, and of the bf16 scan registers for four
waves a SIMD (two workgroups a CU) with next to no spills, what its chunk time was measured with."""
import os
import re

import pytest
from test_isa import CSRC, _asm


def kernels(text):
    """{symbol: (vector registers, spilled registers)} from the code object's metadata."""
    out = {}
    for m in re.finditer(r"- \.agpr_count:.*?\.wavefront_size", text, re.S):
        field = dict(re.findall(r"\.(symbol|vgpr_count|vgpr_spill_count):\s+(\S+)", m.group(0)))
        out[field["symbol"]] = int(field["vgpr_count"]), int(field["vgpr_spill_count"])
    return out


@pytest.mark.parametrize("src", ["kda_conv.hip", "kda_qk_norm.hip", "kda_ssm_decode.hip", "kda_ssm.hip"])
def test_layer_kernel_isa(src, tmp_path):
    text = _asm(os.path.join(CSRC, src), tmp_path)
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)
    found = kernels(text)
    assert found
    for name, (vgprs, spills) in found.items():
        assert spills <= (2 if src == "kda_ssm.hip" else 0), name
        if re.search(r"ssm_kernelIDF16bLi(64ELi\d+ELi2|128ELi\d+ELi1)ELb1ELb[01]ELb0E", name):
            assert vgprs <= 128, name
