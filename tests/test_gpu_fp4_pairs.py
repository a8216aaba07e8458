"""Products by CTA pairs in every tile width, with last tiles that are not full: what surrounds the output stays as it was,
rows that hold no numbers stay by themselves, scale bytes behind the last row count for nothing."""
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb
from fp4_pair_shapes import SHAPES
from test_gpu_fp4 import FORMATS, check_product, dense, operands, quantised

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,bn", SHAPES)
def test_what_surrounds_the_output(M, N, K, bn, fmt):
    a, w = operands(M, N, K, fmt, M + N)
    da, dw = dense(a, fmt), dense(w, fmt)
    want = fb.fp4_gemm(*a, *w, fmt)
    check_product(want, da, dw, K)
    for shift in (8, 1, 4):            # elements: pairs, then places where the pairs do not store
        buf = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[shift:shift + M * N].view(M, N)
        fb.fp4_gemm(*a, *w, fmt, out=out)
        assert bool((buf[:shift] == 7).all()) and bool((buf[shift + M * N:] == 7).all())
        if shift == 8:
            assert torch.equal(out, want)
        else:
            check_product(out, da, dw, K)
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,bn", SHAPES)
def test_rows_that_hold_no_numbers(M, N, K, bn, fmt):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    wt = torch.randn(N, K, generator=g, device="cuda")
    bad_m, bad_n = [1, M // 2, M - 1], [0, N // 2, N - 1]
    for i, m in enumerate(bad_m):
        x[m, (5, K // 2, K - 1)[i]] = (float("inf"), float("nan"), -float("inf"))[i]
    for i, n in enumerate(bad_n):
        wt[n, (K - 1, 3, K // 2)[i]] = (float("nan"), float("inf"), float("nan"))[i]
    a, w = quantised(x, wt, fmt)
    for op, rows in ((a, M), (w, N)):
        flat = op[1].permute(0, 3, 2, 1, 4).reshape(-1, op[1].shape[1] * 4)      # a copy [rows, blocks]
        flat[rows:] = torch.where(torch.arange(flat.shape[1], device="cuda") % 2 == 0, 255, 127).to(torch.uint8)
        op[1].copy_(flat.view(op[1].shape[0], 4, 32, op[1].shape[1], 4).permute(0, 3, 2, 1, 4))
    torch.cuda.synchronize()
    c = fb.fp4_gemm(*a, *w, fmt)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[bad_m], bad[:, bad_n] = True, True
    assert torch.equal(c.isnan(), bad)
    da, dw = dense(a, fmt).nan_to_num(0.0), dense(w, fmt).nan_to_num(0.0)
    check_product(torch.where(bad, (da @ dw.t()).bfloat16(), c), da, dw, K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,bn", SHAPES)
def test_linear_and_its_repeats(M, N, K, bn, fmt):
    """The layer is its two calls, bit for bit, alone, in a row with others and in a graph on a stream of its own."""
    a, w = operands(M, N, K, fmt, N)
    xs = [torch.randn(M, K, device="cuda").bfloat16() for _ in range(2)]
    want = [fb.fp4_gemm(*fb.fp4_quant(x, fmt), *w, fmt) for x in xs]
    for _ in range(4):
        got = [fb.fp4_linear(x, *w, fmt) for x in xs]
        assert all(torch.equal(c, v) for c, v in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = xs[0].clone()
    with torch.cuda.stream(side):
        fb.fp4_linear(x, *w, fmt)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = fb.fp4_linear(x, *w, fmt)
    torch.cuda.synchronize()
    for i in (1, 0):
        x.copy_(xs[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    assert fb.last_device_error() == 0
