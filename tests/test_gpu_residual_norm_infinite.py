"""Infinite factors of the norm: a column that one makes infinite is its row's whole sum, so by the formula the other columns'
h are 0 (a finite number over infinity) and that column's is no number, whatever the row's length is."""
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["post", "column", "token", "post and column"])
@pytest.mark.parametrize("T", [1, 5, 400])
@pytest.mark.parametrize("D", [512, 640, 1288, 6272, 8960])
def test_an_infinite_factor(D, T, what):
    g = torch.Generator(device="cuda").manual_seed(D + T)
    y = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    norm, post, column = torch.ones(D, device="cuda"), None, None
    y[:, 3] = 2.0
    col = 3
    if "post" in what:
        post = torch.ones(D, device="cuda")
        if what == "post":
            post[col] = float("inf")
    gate = None
    if "column" in what:
        gate = torch.ones(D, device="cuda")
        gate[col] = -float("inf")
    if what == "token":
        post = torch.ones(D, device="cuda")
        gate = torch.ones(T, D, device="cuda").bfloat16()
        gate[:, col] = float("inf")
    r, h = fb.residual_norm(y, x, norm, post_w=post, gate=gate)
    z = y.double()
    if post is not None:
        z = z / (z.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * post.double()
    if gate is not None:
        z = z * gate.double()
    want = x.double() + z
    others = torch.arange(D, device="cuda") != col
    assert torch.equal(r[:, col].double(), want[:, col])
    # (half a bf16 step of r, and the fp32 steps before it: at most 2^-19 of the terms)
    off = (r.double() - want)[:, others].abs()
    assert bool((off <= 2.0 ** -8 * want[:, others].abs() + 2.0 ** -19 * (x.double().abs() + z.abs())[:, others]).all())
    assert bool((h[:, others] == 0).all()) and bool(h[:, col].isnan().all())
