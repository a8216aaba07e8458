"""What the few-token MoE layer waits for before a CTA ends after a wait that gave up: the function that keeps its
token copies' barriers, compiled from the kernel's own source and run on the host (no GPU).

A barrier's phases complete in turn, so its last copy is in memory when the phase of parity (copies so far - 1) % 2 has
completed; a barrier without any copy must not be waited for."""
import os
import random
import shutil
import subprocess

import pytest

STAGES = 10


def armed(lines, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    here = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(here)
    exe = str(tmp_path / "armed_phases_dump")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-std=c++17",
                    "--expt-relaxed-constexpr", "-I", os.path.join(root, "include"),
                    "-I", os.path.join(root, "fp8_block_scaled_quant_gb300", "csrc"),
                    "-o", exe, os.path.join(here, "cuda", "armed_phases_dump.cu")],
                   check=True, capture_output=True, timeout=300)
    res = subprocess.run([exe], input="".join(" ".join(map(str, l)) + "\n" for l in lines), capture_output=True,
                         text=True, timeout=120)
    assert res.returncode == 0
    return [tuple(int(v) for v in l.split()) for l in res.stdout.splitlines()]


def test_last_phase_of_every_barrier(tmp_path):
    rng = random.Random(5)
    lines = [[], [0], [3, 3], [9] * 5, [(2 * q) % STAGES for q in range(23)], list(range(STAGES)) * 3 + [0, 1]]
    lines += [[rng.randrange(STAGES) for _ in range(rng.randint(1, 200))] for _ in range(200)]
    got = armed(lines, tmp_path)
    assert len(got) == len(lines)
    for l, (used, parity) in zip(lines, got):
        assert used == sum(1 << s for s in set(l))
        for s in set(l):
            assert (parity >> s) & 1 == (l.count(s) - 1) % 2, (l, s)


def test_every_bulk_copy_of_the_layer_is_waited_for():
    """The barriers that copies complete on are the weight tiles' and the tokens'; both are in the wait before the end."""
    here = os.path.dirname(os.path.abspath(__file__))
    with open(os.path.join(os.path.dirname(here), "fp8_block_scaled_quant_gb300", "csrc", "moe_layer.cu")) as f:
        src = f.read()
    kernel = src[src.index("moe_layer_kernel("):src.index("typedef CUresult")]
    armed_on = {a.split("[")[0] for a in (p.split(",")[0] for p in kernel.split("mbar_arrive_expect_tx(&")[1:])}
    assert armed_on == {"full", "tok_full"}
    end = kernel[kernel.rindex("if (*abort_flag) {"):]
    for name in armed_on:
        assert f"wait(&{name}[" in end, name
