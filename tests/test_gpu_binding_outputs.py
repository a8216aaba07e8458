"""The outputs of the 4-bit calls and the norm are tensors of their own: each has its storage and no more, so that one can be
kept, saved, resized or handed to another stream without the others."""
import io

import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu


def leaves(v):
    return [v] if isinstance(v, torch.Tensor) else [t for x in v if x is not None for t in leaves(x)]


def calls(T):
    x = torch.randn(T, 256, device="cuda").bfloat16()
    one = torch.ones(256, device="cuda")
    q = fb.fp4_quant(x)
    torch.cuda.synchronize()
    return {"quant": lambda: fb.fp4_quant(x), "quant ue8m0": lambda: fb.fp4_quant(x, fb.FP4_UE8M0),
            "norm": lambda: fb.residual_norm(x, x, one), "norm fp8": lambda: fb.residual_norm(x, x, one, quant="fp8"),
            "norm fp4": lambda: fb.residual_norm(x, x, one, quant="fp4"),
            "norm ue8m0": lambda: fb.residual_norm(x, x, one, quant="fp4", scale_fmt=fb.FP4_UE8M0),
            "gemm": lambda: fb.fp4_gemm(*q, *q), "linear": lambda: fb.fp4_linear(x, *q), "dequant": lambda: fb.fp4_dequant(*q)}


NAMES = ["quant", "quant ue8m0", "norm", "norm fp8", "norm fp4", "norm ue8m0", "gemm", "linear", "dequant"]


@pytest.mark.parametrize("T", [0, 1, 7, 3000])
@pytest.mark.parametrize("name", NAMES)
def test_each_output_has_its_storage(name, T):
    out = leaves(calls(T)[name]())
    assert out and all(t.storage_offset() == 0 and t.is_contiguous() and not t.requires_grad for t in out)
    assert all(t.untyped_storage().nbytes() == t.numel() * t.element_size() for t in out)
    assert all(t.device == torch.device("cuda", torch.cuda.current_device()) for t in out)
    at = [t.untyped_storage().data_ptr() for t in out if t.numel()]
    assert len(set(at)) == len(at) and all(p % 256 == 0 for p in at)


@pytest.mark.parametrize("name", NAMES)
def test_an_output_grows_without_the_others(name):
    out = leaves(calls(7)[name]())
    kept = [t.view(torch.uint8).clone() for t in out]
    for i, t in enumerate(out):
        t.resize_(t.numel() * 4)
        t.view(torch.uint8)[kept[i].numel():].fill_(0xA5)
        now = [u.view(torch.uint8).flatten()[:k.numel()] for u, k in zip(out, kept)]
        assert all(torch.equal(a, k.flatten()) for a, k in zip(now, kept))
    f = io.BytesIO()
    torch.save(out[0], f)
    assert f.tell() < out[0].numel() * out[0].element_size() + 4096


def test_memory_is_given_back_with_each_output():
    make = calls(7)["norm fp4"]
    make()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    r, h = make()
    sizes = [-(-t.numel() * t.element_size() // 512) * 512 for t in [r, *h]]
    assert torch.cuda.memory_allocated() - before == sum(sizes)
    del h
    assert torch.cuda.memory_allocated() - before == sizes[0]
    del r
    assert torch.cuda.memory_allocated() == before


def test_outputs_in_inference_mode_and_on_a_stream():
    c = calls(7)
    side = torch.cuda.Stream()
    with torch.inference_mode(), torch.cuda.stream(side):
        r, h = c["norm"]()
        assert r.is_inference() and not r.requires_grad
        r.record_stream(torch.cuda.current_stream())
    side.synchronize()
    want, _ = c["norm"]()
    assert torch.equal(r, want) and not want.is_inference()
    want.requires_grad_().float().sum().backward()
    assert torch.equal(want.grad, torch.ones_like(want))
