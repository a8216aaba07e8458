"""fp4_linear from several Python threads on one stream: its quantised activations lie in a workspace that the calls of the
stream share, so the two launches of a call must follow each other, with no other call's in between."""
import threading

import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own_stream", [False, True])
@pytest.mark.parametrize("M,N,K", [(8, 512, 1024), (40, 640, 2048), (200, 328, 512)])
def test_threads_share_a_stream(M, N, K, own_stream):
    g = torch.Generator(device="cuda").manual_seed(M)
    w = fb.fp4_quant(torch.randn(N, K, generator=g, device="cuda"))
    xs = [torch.randn(M, K, generator=g, device="cuda").bfloat16() for _ in range(4)]
    torch.cuda.synchronize()
    want = [fb.fp4_gemm(*fb.fp4_quant(x), *w) for x in xs]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if own_stream else torch.cuda.default_stream()
    off, start = [], threading.Barrier(len(xs))

    def work(i):
        with torch.cuda.stream(stream):
            start.wait()
            got = [fb.fp4_linear(xs[i], *w) for _ in range(400)]
            stream.synchronize()
            off.append(sum(not torch.equal(c, want[i]) for c in got))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert off == [0] * len(xs), off
    assert fb.last_device_error() == 0
