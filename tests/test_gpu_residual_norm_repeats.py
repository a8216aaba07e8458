"""The norm gives the same bits again: alone, behind a call on other tensors with nothing waited for in between, and in a
graph. Sizes for each of its kernels: few tokens, a block to a token, and from token to token (more than two tokens to an
SM, a post norm, no gate by token)."""
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu


def bits(v):
    return [t.clone().view(torch.uint8) for t in ([v[0]] + list(v[1] if isinstance(v[1], tuple) else [v[1]])) if t is not None]


@pytest.mark.parametrize("out", [(None, 0), ("fp8", 0), ("fp8", 1), ("fp4", fb.FP4_E4M3), ("fp4", fb.FP4_UE8M0)])
@pytest.mark.parametrize("T,D,gate", [(3, 1024, "column"), (500, 5120, "token"), (2000, 7168, "column"), (311, 640, None)])
def test_the_same_bits(T, D, gate, out):
    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        y, x = rnd(T, D).bfloat16(), (4 * rnd(T, D)).bfloat16()
        y[T // 2] = -x[T // 2]                 # a row whose terms nearly cancel: the long way round
        k = {None: None, "column": 1 + 0.1 * rnd(D), "token": rnd(T, D).bfloat16()}[gate]
        norm, post = 1 + 0.1 * rnd(D), 4 + 0.01 * rnd(D)

        def call():
            r, h = fb.residual_norm(y, x, norm, post_w=post, gate=k, quant=out[0], scale_fmt=out[1])
            if out[0] == "fp4":            # (scale bytes behind the last row are not written)
                s = h[1].permute(0, 3, 2, 1, 4).reshape(-1, h[1].shape[1] * 4)[:T]
                h = (h[0], s, h[2])
            return r, h

        return call

    one, other = make(1), make(2)
    torch.cuda.synchronize()
    want = bits(one())
    torch.cuda.synchronize()
    for turn in range(10):
        one()
        other()
        got = one()
        if turn % 2:
            torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bits(got), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        one()
        other()
        kept = one()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bits(kept), want))
    assert fb.last_device_error() == 0
