"""The norm around a block of so many tokens that a block of threads goes from token to token: every output type, rows
that end its loop at different turns, tokens that take the long way among ones that do not, outputs in place. Tolerances
as in test_gpu_residual_norm.py, whose checks these are."""
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb
import test_gpu_residual_norm as norm

pytestmark = pytest.mark.gpu
SHAPES = [(305, 7168), (457, 8192), (913, 6144), (1400, 2048), (6000, 128), (2433, 1536), (700, 5120)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("gate", [None, "column"])
def test_outputs(T, D, gate):
    norm.test_bf16(T, D, True, gate, 0.7, True)
    norm.test_fp8(T, D, True, gate, 1.0, False)
    norm.test_fp8(T, D, True, gate, 1.3, True)
    norm.test_fp4(T, D, True, gate, 1.0, fb.FP4_UE8M0)
    norm.test_fp4(T, D, True, gate, 1.0, fb.FP4_E4M3)


@pytest.mark.parametrize("T,D", [(1000, 7168), (2000, 512)])
@pytest.mark.parametrize("quant", [None, "fp8"])
def test_tokens_are_their_own_affair(T, D, quant):
    """Tokens of zeros, far sizes, a NaN, an infinity, and ones whose terms cancel, between ordinary ones: the ordinary
    ones' outputs stay bit for bit, the finite others follow the formula."""
    a = norm.make(T, D, 5, True, "column")
    g = torch.Generator(device="cuda").manual_seed(2)
    kind = torch.randint(0, 12, (T,), generator=g, device="cuda")
    odd = norm.make(T, D, 5, True, "column")
    z = norm.formula({**a, "x": torch.zeros_like(a["y"])}, 1.0)[0]
    odd["y"][kind == 1], odd["x"][kind == 1] = 0, 0
    odd["y"][kind == 2] *= 2.0 ** 60
    odd["x"][kind == 3] *= 2.0 ** 50
    odd["y"][kind == 4] *= 2.0 ** -90
    odd["x"][kind == 4] = 0
    odd["x"][kind == 5] = (-z * (1 + 0.01 * torch.randn(T, D, generator=g, device="cuda"))).bfloat16()[kind == 5]
    odd["y"][kind == 6, 3] = float("nan")
    odd["x"][kind == 7, D - 1] = float("inf")
    same, bad = (kind == 0) | (kind > 7), (kind == 6) | (kind == 7)
    want, got = fb.residual_norm(**a, eps=norm.EPS, quant=quant), fb.residual_norm(**odd, eps=norm.EPS, quant=quant)
    flat = lambda t: [t[0], t[1]] if quant is None else [t[0], t[1][0].view(torch.uint8), t[1][1]]  # noqa: E731
    for u, v in zip(flat(got), flat(want)):
        assert torch.equal(u[same], v[same])
    if quant is None:
        wr, er, wh, eh = norm.formula(odd, 1.0)
        norm.close(got[0][~bad], wr[~bad], er[~bad])
        norm.close(got[1][~bad], wh[~bad], eh[~bad])
    assert bool(got[0][kind == 6].isnan().any(1).all())
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("name", ["x", "y"])
def test_in_place(name):
    a = norm.make(1234, 2048, 8, True, "column")
    want = fb.residual_norm(**a, quant="fp8")
    got = fb.residual_norm(**a, quant="fp8", r=a[name])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1][1], want[1][1])
    assert torch.equal(got[1][0].view(torch.uint8), want[1][0].view(torch.uint8))


def test_captured():
    a = norm.make(777, 7168, 9, True, "column")
    want = fb.residual_norm(**a)
    y, x = a["y"].clone(), a["x"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            first = fb.residual_norm(**{**a, "y": y, "x": x})
            second = fb.residual_norm(**{**a, "y": first[1], "x": first[0]})
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], want[0]) and torch.equal(first[1], want[1])
    again = fb.residual_norm(**{**a, "y": want[1], "x": want[0]})
    assert torch.equal(second[0], again[0]) and torch.equal(second[1], again[1])
