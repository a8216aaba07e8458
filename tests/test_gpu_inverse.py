"""The norm's reciprocals stay within their bounds, and its e4m3 scale is the IEEE quotient, for every fp32 input (about 6e9
values, compiled from tests/cuda/inverse_check.cu around the library's own header). The bounds: Newton's step squares the
estimate's error, which leaves the roundings of the step."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp8_block_scaled_quant_gb300", "csrc")


def test_reciprocals_and_scale_over_every_input(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "inverse_check")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-I", CSRC, "-o", exe,
                    os.path.join(HERE, "cuda", "inverse_check.cu")], check=True, capture_output=True, timeout=300)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    lines = res.stdout.strip().splitlines()
    assert len(lines) == 3 and all(ln.endswith(" outside 0") for ln in lines), res.stdout + res.stderr
    assert res.returncode == 0, res.stdout
