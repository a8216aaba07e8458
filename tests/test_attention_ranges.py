"""How the latent attention splits its units (key tiles, and one per item) over CTA pairs: the function compiled from
the kernel's own source, run on the host (no GPU).

Each pair takes the units from its first one to the next pair's. The ranges have to cover every unit once and stay
inside them: a pair that took a unit that is not there would look for an item that no plan names. A batch without any
key has no units, and then every range is empty."""
import os
import shutil
import subprocess

import pytest


def first_units(cases, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    here = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(here)
    exe = str(tmp_path / "attention_ranges_dump")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-std=c++17",
                    "--expt-relaxed-constexpr", "-I", os.path.join(root, "include"),
                    "-I", os.path.join(root, "fp8_block_scaled_quant_gb300", "csrc"),
                    "-o", exe, os.path.join(here, "cuda", "attention_ranges_dump.cu")],
                   check=True, capture_output=True, timeout=300)
    res = subprocess.run([exe], input="".join(f"{u} {p}\n" for u, p in cases), capture_output=True, text=True,
                         timeout=120)
    lines = [[int(v) for v in line.split()] for line in res.stdout.splitlines()]
    assert res.returncode == 0 and len(lines) == len(cases)
    return lines


def test_ranges_cover_the_units_once(tmp_path):
    cases = [(u, p) for p in (1, 2, 66, 76, 96)
             for u in sorted({0, 1, 2, p - 1, p, p + 1, 2 * p - 1, 2 * p, 1000, 12345, (1 << 20) + 7, (1 << 30) - 1})]
    for (units, pairs), at in zip(cases, first_units(cases, tmp_path)):
        assert len(at) == pairs + 1 and at[0] == 0 and at[-1] == units, (units, pairs, at)
        sizes = [b - a for a, b in zip(at, at[1:])]
        assert min(sizes) >= 0 and max(sizes) <= -(-units // pairs), (units, pairs, at)
        if units >= pairs:   # as the rows' parts are looked up: the largest q with units q / pairs <= u
            assert at == [units * q // pairs for q in range(pairs + 1)]
        else:
            assert at == [min(q, units) for q in range(pairs + 1)]
