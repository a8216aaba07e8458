"""Which kernel the 4-bit product takes, from the library's own rules compiled for the host (no GPU): the sizes that the GPU
tests use for the CTA pairs reach them, in every tile width, and what the pairs' stores cannot do goes elsewhere."""
import os
import shutil
import subprocess

import pytest

from fp4_pair_shapes import SHAPES

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SMS = 152


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("plans") / "fp4_plan_dump")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-std=c++17", "--expt-relaxed-constexpr",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "fp8_block_scaled_quant_gb300", "csrc"),
                    "-o", exe, os.path.join(HERE, "cuda", "fp4_plan_dump.cu")], check=True, capture_output=True, timeout=300)

    def ask(shapes):
        text = "".join(f"{m} {n} {k} {aligned} {SMS}\n" for m, n, k, aligned in shapes)
        res = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert res.returncode == 0
        return [ln.split() for ln in res.stdout.splitlines()]

    return ask


def test_the_pairs_sizes_reach_every_tile_width(plans):
    got = plans([(m, n, k, 1) for m, n, k, _ in SHAPES])
    assert [p[:2] for p in got] == [["pairs", str(bn)] for *_, bn in SHAPES]
    assert {bn for *_, bn in SHAPES} == {128, 256, 384}
    assert all(m % 128 and n % 128 for m, n, *_ in SHAPES)


def test_other_rows_and_places_go_to_the_few_token_kernel(plans):
    """Rows that are no multiple of 16 bytes, or an output that does not begin at one."""
    for m, n, k, _ in SHAPES:
        rows, place = plans([(m, n + 1, k, 1), (m, n, k, 0)])
        assert rows[0] == "few" and place[0] == "few"


def test_splits_are_within_a_cluster_and_cover_k(plans):
    shapes = [(m, n, k, 1) for m in (1, 2, 8, 16, 17, 32, 33, 48, 64, 100) for n in (1, 128, 1000, 2112, 7168, 24576)
              for k in (128, 256, 640, 2048, 7168, 18432, 1 << 20)]
    for (m, n, k, _), p in zip(shapes, plans(shapes)):
        if p[0] == "few":
            stages = -(-k // 256)
            assert 1 <= int(p[2]) <= 8 and (int(p[2]) == 1 or 2 * int(p[2]) <= stages), (m, n, k, p)
        fused = int(p[-1])
        assert not fused or (m <= 16 and m * k <= (8192 if m == 1 else 4096)), (m, n, k, p)
