"""The binding's workspaces and captured graphs: a graph keeps the addresses it was captured with, so their buffers
stay allocated whatever later calls need; a buffer made during a capture is filled by that graph and shared with no
other call."""
import types

import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb


class Host:
    """The cache on host tensors, with a capture switched on and off by the test (`capturing`: its number)."""

    def __init__(self, monkeypatch):
        self.capturing = False
        monkeypatch.setattr(fb, "_ws_graph", {})
        monkeypatch.setattr(fb, "_capture_id", lambda stream: self.capturing)
        monkeypatch.setattr(fb, "_ws_cache", {})
        monkeypatch.setattr(fb, "_ws_captured", {})
        monkeypatch.setattr(fb, "_capturing", lambda on_gpu: bool(self.capturing))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=7))
        self.t = torch.zeros(1)

    def scratch(self, nbytes, capturing=False):
        self.capturing = capturing
        return fb._scratch(None, nbytes, self.t, 7, "op", 256)

    def workspace(self, nbytes, capturing=False):
        self.capturing = capturing
        return fb.workspace(nbytes, torch.device("cpu"), "op")


def alive(at):
    return any(b.data_ptr() <= at < b.data_ptr() + b.numel() for b in fb._ws_captured.values())


def test_a_captured_buffer_outlives_a_larger_one(monkeypatch):
    h = Host(monkeypatch)
    first, room, _ = h.scratch(1000)
    assert h.scratch(1000, capturing=True)[0] == first and room == 1000     # warmed up: the same buffer
    larger, _, _ = h.scratch(1 << 20)
    assert larger != first and alive(first)
    assert h.scratch(500)[0] == larger                                      # and the larger one serves from now on


def test_a_captured_workspace_outlives_a_larger_one(monkeypatch):
    h = Host(monkeypatch)
    first = h.workspace(1000).data_ptr()
    assert h.workspace(900, capturing=True).data_ptr() == first
    assert h.workspace(1 << 20).data_ptr() != first and alive(first)


def test_buffers_of_no_graph_are_given_back(monkeypatch):
    h = Host(monkeypatch)
    for n in (1000, 10000, 100000):
        h.scratch(n)
    assert len(fb._ws_cache) == 1 and not fb._ws_captured


@pytest.mark.parametrize("take", ["scratch", "workspace"])
def test_a_buffer_made_in_a_capture_serves_that_capture_alone(monkeypatch, take):
    """Its fill runs once in each of that graph's replays: the graph's other calls share it, another graph or an eager
    call may not."""
    h = Host(monkeypatch)
    tensor = lambda got: got[2] if take == "scratch" else got
    at = lambda got: got[0] if take == "scratch" else got.data_ptr()
    first = getattr(h, take)(4096, capturing=11)
    assert not tensor(first)[:512].any() and not fb._ws_cache and not fb._ws_captured
    assert at(getattr(h, take)(3000, capturing=11)) == at(first)
    assert at(getattr(h, take)(1 << 20, capturing=11)) != at(first)
    other = getattr(h, take)(4096, capturing=12)
    eager = getattr(h, take)(4096)
    assert len({at(first), at(other), at(eager)}) == 3
    kept, = fb._ws_cache.values()
    assert not kept.any() and at(getattr(h, take)(4096, capturing=13)) == at(eager)


class OnGpu:
    """Stands for a tensor of GPU 0, as far as a workspace's check looks."""

    def get_device(self):
        return 0


def test_a_given_workspace_is_checked():
    """A kernel would write to whatever address it is given: host memory and strided views are refused, and the size is
    counted in bytes."""
    for bad, t in ((torch.zeros(4096, dtype=torch.uint8), OnGpu()), (torch.zeros(8192, dtype=torch.uint8)[::2],
                                                                     torch.zeros(1))):
        with pytest.raises(fb.Fp8BlkError):
            fb._scratch(bad, 1000, t, 7, "op", 256)
    ws = torch.zeros(1024, dtype=torch.int32)
    assert fb._scratch(ws, 1000, torch.zeros(1), 7, "op", 256)[:2] == (ws.data_ptr(), 4096)


@pytest.mark.gpu
def test_a_host_workspace_is_refused():
    a, b = moe(2, 512, 256, 32, 7), attention(1, 16, 20, 8)
    (w1, w3, w2), (s1, s3, s2) = a["w"], a["s"]
    with pytest.raises(fb.Fp8BlkError):
        fb.moe_layer(a["x"], a["gate"], w1, s1, w3, s3, w2, s2, topk=4, ws=torch.zeros(1 << 25, dtype=torch.uint8))
    with pytest.raises(fb.Fp8BlkError):
        fb.mla_attention(b["q"], b["pe"], b["cache"], b["table"], b["lens"], 0.07,
                         ws=torch.zeros(1 << 25, dtype=torch.uint8))


def moe(T, dim, inter, E, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    w = [(n(E * r, c) * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for r, c in ((inter, dim), (inter, dim), (dim, inter))]
    s = [torch.full((t.shape[0] // 128, t.shape[1] // 128), 2e-4, device="cuda") for t in w]
    return dict(x=n(T, dim).bfloat16(), gate=(n(E, dim) * dim ** -0.5).bfloat16(), w=w, s=s)


def run_moe(a, out=None):
    (w1, w3, w2), (s1, s3, s2) = a["w"], a["s"]
    return fb.moe_layer(a["x"], a["gate"], w1, s1, w3, s3, w2, s2, topk=4, out=out)


def attention(B, H, n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    pages = -(-n // 64)
    return dict(q=r(B, H, 512), pe=r(B, H, 64), cache=r(B * pages, 64, 576),
                table=torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages),
                lens=torch.full((B,), n, dtype=torch.int32, device="cuda"))


def run_attention(a, out=None):
    return fb.mla_attention(a["q"], a["pe"], a["cache"], a["table"], a["lens"], 0.07, out=out)


def linear(M, N, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return dict(x=torch.randn(M, K, generator=g, device="cuda").bfloat16(),
                w=fb.weight_quant(torch.randn(N, K, generator=g, device="cuda")))


def run_linear(a, out=None):
    return fb.linear(a["x"], *a["w"], out=out)


CASES = {
    "moe_layer": (run_moe, lambda: moe(2, 512, 256, 32, 1), lambda: moe(32, 2048, 512, 64, 2)),
    "mla_attention": (run_attention, lambda: attention(1, 16, 700, 3), lambda: attention(64, 128, 300, 4)),
    "linear": (run_linear, lambda: linear(8, 1024, 2048, 5), lambda: linear(700, 7000, 7168, 6)),
}


def ready(stream):
    stream.wait_stream(torch.cuda.current_stream())
    return torch.cuda.stream(stream)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_a_graph_survives_a_larger_call_on_its_stream(name):
    run, small, large = CASES[name]
    a, b = small(), large()
    ref, out = run(a), torch.empty_like(run(a))
    stream = torch.cuda.Stream()
    with ready(stream):
        run(a)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run(a, out)
        want = run(b)
        # What the allocator may now hand out again is someone else's.
        others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 20, 1 << 21, 1 << 23)
                  for _ in range(8)]
        for _ in range(2):
            out.zero_()
            graph.replay()
        again = run(b)
    stream.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    assert torch.equal(want.view(torch.int16), again.view(torch.int16))
    assert all(bool((t == 0x5A).all()) for t in others)
    assert fb.last_device_error() == 0


@pytest.mark.gpu
def test_capture_id():
    assert fb._capture_id(torch.cuda.current_stream().cuda_stream) == 0
    seen, x = [], torch.zeros(1, device="cuda")
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(2):
                x += 1
                seen.append(fb._capture_id(torch.cuda.current_stream().cuda_stream))
    assert seen[0] == seen[1] != seen[2] == seen[3] and 0 not in seen


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_calls_of_one_capture_share_their_buffer(name):
    """Warmed up on the default stream, captured on the capture's own: one buffer, filled once in a replay."""
    run, small, _ = CASES[name]
    a = small()
    ref = run(a)
    outs = [torch.empty_like(ref) for _ in range(3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    before = dict(fb._ws_graph)
    with torch.cuda.graph(graph):
        held = []
        for o in outs:
            run(a, o)
            new = [v[1].data_ptr() for k, v in fb._ws_graph.items() if v is not before.get(k)]
            held.append(new)
    assert held[0] == held[1] == held[2] and len(held[0]) <= 1
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), ref.view(torch.int16))
    assert fb.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_graphs_captured_without_a_call_before(name):
    """Two graphs of a stream that no call ran on: each brings its own zeros, in whatever order they are replayed, and
    so does a call on that stream."""
    run, small, _ = CASES[name]
    a = small()
    ref = run(a)
    outs = [torch.empty_like(ref) for _ in range(2)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with ready(stream):
        graphs = []
        for o in outs:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                run(a, o)
        got = run(a)
        for k in (1, 0, 1):
            outs[k].zero_()
            graphs[k].replay()
    stream.synchronize()
    for o in (*outs, got):
        assert torch.equal(o.view(torch.int16), ref.view(torch.int16))
    assert fb.last_device_error() == 0
