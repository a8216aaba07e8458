"""Loads of the 4-bit and norm kernels and the dependency wait, by the sources (no GPU). What a kernel that starts early
reads before its wait may still be the previous kernel's to write. The compiler keeps plain loads and volatile asm with a
memory clobber behind the wait; loads declared read-only it may move across."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_quant_gb300", "csrc")
FILES = ["fp4.cuh", "fp4_quant.cu", "gemm_fp4.cu", "residual_norm.cu"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_no_load_is_declared_read_only(name):
    src = source(name)
    assert not re.findall(r"\.nc\b|__ldg\b|__ldc[sgav]\b|__restrict__", src)
    # (the helpers of ptx.cuh that these use, too)
    for text in (src, source("ptx.cuh")):
        for load in re.findall(r"asm[^;]*?\(\s*\"ld\.global.*?\);", text, re.S):
            assert load.startswith("asm volatile") and load.rstrip(");").rstrip().endswith('"memory"'), load


def test_the_wait_is_a_barrier_to_the_compiler():
    assert 'asm volatile("griddepcontrol.wait;" ::: "memory")' in source("ptx.cuh")
