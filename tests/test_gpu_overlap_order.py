"""Calls in an order that the rule on overlap allows: an operand written by one call is a later product's weight, with
early calls and one ordering call in between."""
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("M", [16, 100])
@pytest.mark.parametrize("order", ["quant", "dequant", "torch"])
def test_norm_into_a_weight(M, order):
    """The norm runs on all SMs for tens of microseconds, the two after it start beside it; the ordering call holds the
    product back until the operand is there."""
    fmt, T, D = fb.FP4_UE8M0, 4000, 6144
    g = torch.Generator(device="cuda").manual_seed(M)
    keys = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    ones = torch.ones(D, device="cuda")
    small = [torch.randn(4, 1024, generator=g, device="cuda").bfloat16() for _ in range(3)]
    one = torch.ones(1024, device="cuda")
    a = fb.fp4_quant(torch.randn(M, D, generator=g, device="cuda").bfloat16(), fmt)
    tiny = fb.fp4_quant(small[0], fmt)
    torch.cuda.synchronize()
    want = None
    for turn in range(6):
        _, w = fb.residual_norm(keys, None, ones, post_w=ones, quant="fp4", scale_fmt=fmt)
        fb.residual_norm(small[0], None, one)
        fb.residual_norm(small[1], None, one)
        if want is None:
            torch.cuda.synchronize()
        elif order == "quant":
            fb.fp4_quant(small[2], fmt)
        elif order == "dequant":
            fb.fp4_dequant(*tiny, fmt)
        else:
            small[2].add_(0)
        fb.residual_norm(small[2], None, one)
        c = fb.fp4_gemm(*a, *w, fmt)
        torch.cuda.synchronize()
        if want is None:
            want = c.clone()
        assert torch.equal(bits(c), bits(want))
        w[0].fill_(0x77), w[1].fill_(0)      # what a product that came too early would read
        torch.cuda.synchronize()
        del w
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("M", [1, 8, 300])
def test_quantised_just_before(M):
    """A weight that was quantised on the way, finished before it is multiplied by; the activations straight after."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, 1024, generator=g, device="cuda").bfloat16()
    w = torch.randn(520, 1024, generator=g, device="cuda")
    both = [fb.fp4_quant(t) for t in (w, x)]
    torch.cuda.synchronize()
    want = fb.fp4_gemm(*both[1], *both[0])
    for _ in range(5):
        q = fb.fp4_quant(w)
        assert torch.equal(bits(fb.fp4_gemm(*fb.fp4_quant(x), *q)), bits(want))      # (the activations' call orders)
        q = fb.fp4_quant(w)
        torch.cuda.synchronize()
        assert torch.equal(bits(fb.fp4_linear(x, *q)), bits(want))
