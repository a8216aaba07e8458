"""The norm around a block where the residual and the block's output nearly cancel, and where their sums leave fp32's
comfortable range: the square sum of r is then taken from r itself. Tolerances as in test_gpu_residual_norm.py."""
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb
from test_gpu_residual_norm import EPS, close, formula, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 400])
@pytest.mark.parametrize("D", [384, 7168, 1000])
@pytest.mark.parametrize("left", [0.5, 0.05, 0.001])
def test_nearly_cancelling(T, D, left):
    """x is minus the normed and gated y but for a share `left`: what is left has to be normed as exactly as it stands."""
    a = make(T, D, D, True, "column")
    _, _, z, _ = formula({**a, "x": None, "norm_w": torch.ones(D, device="cuda")}, 1.0)
    z = formula({**a, "x": torch.zeros_like(a["y"])}, 1.0)[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    a["x"] = (-z * (1 + left * torch.randn(T, D, generator=g, device="cuda"))).bfloat16()
    r, h = fb.residual_norm(**a, eps=EPS)
    wr, er, wh, eh = formula(a, 1.0)
    close(r, wr, er)
    close(h, wh, eh)


@pytest.mark.parametrize("T", [2, 400])
@pytest.mark.parametrize("y_exp,x_exp", [(60, 0), (0, 60), (-100, 0), (0, -100), (50, 50), (-70, -70), (-70, 40), (100, 3)])
def test_far_ranges(T, y_exp, x_exp):
    a = make(T, 512, 3, True, "token")
    a["y"], a["x"] = a["y"] * 2.0 ** y_exp, a["x"] * 2.0 ** x_exp
    r, h = fb.residual_norm(**a, eps=EPS)
    wr, er, wh, eh = formula(a, 1.0)
    close(r, wr, er)
    close(h, wh, eh)
