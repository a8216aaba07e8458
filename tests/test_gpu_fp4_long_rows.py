"""Quantisation of rows that a block does not hold in registers (512 threads of six passes have 49152 columns): it reads them
again for the codes. The amax of a row may lie in either part. Against the rule bit for bit, as the shorter rows."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb
from test_gpu_fp4 import FORMATS, check_quant, random_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 49152), (2, 49280), (1, 57344), (3, 65664), (1, 131200)])
@pytest.mark.parametrize("top", ["first", "last", "none"])
def test_long_rows(M, K, fmt, top):
    x = random_rows(M, K, K)
    if top != "none":
        x[:, 7 if top == "first" else K - 3] = 4096.0
    x = x.cuda()
    check_quant(x, fmt, fb.fp4_quant(x, fmt))
    f = (x.float() * 1.2345).contiguous()
    check_quant(f, fmt, fb.fp4_quant(f, fmt))
    wide = torch.zeros(M, K + 72, device="cuda", dtype=torch.bfloat16)
    wide[:, 8:K + 8] = x
    check_quant(wide[:, 8:K + 8], fmt, fb.fp4_quant(wide[:, 8:K + 8], fmt))     # rows at 16, not at 32 bytes


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("where", [3, 49151, 49152, 49279])
def test_a_long_row_that_is_not_finite(fmt, where):
    x = random_rows(2, 49280, 1)
    x[1, where] = float("nan")
    x = x.cuda()
    got = fb.fp4_quant(x, fmt)
    check_quant(x, fmt, got)
    back = fb.fp4_dequant(*got, fmt)
    bad = back.isnan().cpu().numpy()
    want = np.zeros_like(bad)
    if fmt == fb.FP4_E4M3:
        want[1] = True
    else:
        want[1, where // 32 * 32:where // 32 * 32 + 32] = True
    assert np.array_equal(bad, want)
