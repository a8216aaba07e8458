"""Products of 4-bit matrices whose row scales, multiplied with each other, would leave fp32's range, while the results do
not: rows of very small numbers, and rows of very large ones that meet only zeros.

Tolerance: the one of a product (half a bf16 step, 2^-8 of the value; the sum, (K / 64 + 2) 2^-21 of the sum of the products'
sizes, the two scales included), and what rounding to subnormal numbers adds: half of bf16's last step, 2^-134, and of
fp32's, 2^-150."""
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb
from test_gpu_fp4 import dense, quantised

pytestmark = pytest.mark.gpu
FMT = fb.FP4_E4M3
# (tokens: quantised inside the product; a cluster's, without and with a split of K; pairs)
SHAPES = [(1, 300, 512), (9, 256, 2048), (24, 2112, 512), (300, 520, 512), (1300, 1032, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("small,large", [(-64, -64), (-100, -30), (-20, -105), (-110, 40), (60, -110), (-70, 100), (50, 60)])
def test_far_scales(M, N, K, small, large):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda") * 2.0 ** small
    wt = torch.randn(N, K, generator=g, device="cuda") * 2.0 ** large
    a, w = quantised(x.bfloat16(), wt, FMT)
    da, dw = dense(a, FMT), dense(w, FMT)
    want, size = da @ dw.t(), da.abs() @ dw.abs().t()
    tol = 2.0 ** -8 * want.abs() + (K // 64 + 2) * 2.0 ** -21 * size + 2.0 ** -134 + 2.0 ** -150
    for c in (fb.fp4_gemm(*a, *w, FMT), fb.fp4_linear(x.bfloat16(), *w, FMT)):
        bad = (c.double() - want).abs() > tol
        assert not bad.any(), (int(bad.sum()), c[bad][:3], want[bad][:3])


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_large_rows_that_meet_zeros(M, N, K):
    """Every product of the row is 0, whatever the scales' product would be; a row that is not finite stays so."""
    x = torch.zeros(M, K, device="cuda").bfloat16()
    wt = torch.zeros(N, K, device="cuda")
    x[:, 3] = 2.0 ** 100
    wt[:, K - 5] = -(2.0 ** 90)
    a, w = quantised(x, wt, FMT)
    assert float(a[2][0]) * float(w[2][0]) > 3.5e38
    for c in (fb.fp4_gemm(*a, *w, FMT), fb.fp4_linear(x, *w, FMT)):
        assert bool((c == 0).all())
    x[M // 2, 0] = float("inf")
    wt[N // 3, 0] = float("nan")
    a, w = quantised(x, wt, FMT)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[M // 2], bad[:, N // 3] = True, True
    for c in (fb.fp4_gemm(*a, *w, FMT), fb.fp4_linear(x, *w, FMT)):
        assert torch.equal(c.isnan(), bad) and bool((c[~bad] == 0).all())
