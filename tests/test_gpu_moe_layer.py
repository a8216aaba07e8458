"""The few-token MoE layer in one kernel, against the formula in 64 bits.

The reference quantises x exactly as the rule says (fp32 scale and quotient),
takes the expert products in 64 bits, quantises u by the rule and rounds
nothing else. u = silu(h1) h3 comes from fp32 sums of dim products on the GPU,
within e_h = 2^-17 of |w1| . |xq| (128-term tensor-core partials, promoted in
fp32), so an element of u near the border of two e4m3 codes may take the other
one, and a block's scale may move by a unit in the last place. Tolerance per
element of y: its bf16 rounding 2^-8 |y|; fp32 sums, 2^-17 of
sum_j g_j |w2| . |uq|; and the code changes: one code step (1/8 of the value,
the spacing of e4m3) of at most 8 elements of u among the expert rows that feed
the element, each moving y by g |w2 u| / 8, bounded with the largest |w2 u| of
the row. Over the whole output the error's norm is the bf16 rounding's
1.66e-3; 3e-3 is allowed (a wrong expert, scale or missing block of 128
columns among 16 moves it by 0.1 and more)."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu


def pow2_up(s):
    m, e = torch.frexp(s)
    return torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))


def codes(v, ue8m0):
    """(values of the e4m3 codes, scales) of the rule on v [rows, K], fp32 in, 64-bit out."""
    b = v.float().unflatten(-1, (-1, 128))
    s = b.abs().amax(-1, keepdim=True).clamp(min=1e-4)
    s = s / torch.full_like(s, 448.0)
    s = pow2_up(s) if ue8m0 else s
    return ((b / s).to(torch.float8_e4m3fn).double() * s.double()).flatten(-2)


def make(T, dim, inter, E, ns, seed, bias=False, ue8m0=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    K = E + ns
    a = dict(x=n(T, dim).bfloat16(), gate_w=(n(E, dim) * dim ** -0.5).bfloat16(),
             gate_bias=0.1 * n(E) if bias else None)
    for name, r, c in (("w1", inter, dim), ("w3", inter, dim), ("w2", dim, inter)):
        a[name] = (n(K * r, c) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        s = 2e-4 * (0.5 + torch.rand((K * r // 128, c // 128), generator=g, device="cuda"))
        a[name + "_s"] = pow2_up(s) if ue8m0 else s
    return a


def dense(a, name, e, n):
    q, s = a[name], a[name + "_s"]
    k = q.shape[1]
    return (q[e * n:(e + 1) * n].double().view(n // 128, 128, k // 128, 128) *
            s[e * n // 128:(e + 1) * n // 128].double()[:, None, :, None]).view(n, k)


def reference(a, idx, w, ns, ue8m0):
    """(y, tolerance) in 64 bits for a given routing."""
    T, dim = a["x"].shape
    inter, E = a["w2"].shape[1], a["gate_w"].shape[0]
    xq = codes(a["x"], ue8m0)
    y = torch.zeros(T, dim, dtype=torch.float64, device="cuda")
    fp, flips = torch.zeros_like(y), torch.zeros_like(y)
    for e in sorted(set(idx.flatten().tolist())) + list(range(E, E + ns)):
        if e < E:
            t, j = (idx == e).nonzero(as_tuple=True)
            wt = w[t, j].double()
        else:
            t, wt = torch.arange(T, device="cuda"), torch.ones(T, dtype=torch.float64, device="cuda")
        h = xq[t] @ dense(a, "w1", e, inter).t()
        u = codes(h * torch.sigmoid(h) * (xq[t] @ dense(a, "w3", e, inter).t()), ue8m0)
        w2 = dense(a, "w2", e, dim)
        y[t] += wt[:, None] * (u @ w2.t())
        fp[t] += wt[:, None] * (u.abs() @ w2.abs().t())
        big = (u.abs()[:, None, :] * w2.abs()[None]).amax(-1) if len(t) * dim * inter < 1 << 27 else \
            u.abs().amax(-1)[:, None] * w2.abs().amax(-1)[None]
        flips[t] = torch.maximum(flips[t], wt[:, None] * big)
    return y, 2.0 ** -8 * y.abs() + 2.0 ** -17 * fp + flips


def routing(a, topk, G, TG, score, scale, normalize):
    """(ids, weights, gap) of the gate in 64 bits; gap: the least distance of a selected key from the next one."""
    T, E = a["x"].shape[0], a["gate_w"].shape[0]
    logits = a["x"].double() @ a["gate_w"].double().t()
    s = torch.sigmoid(logits) if score == fb.SCORE_SIGMOID else torch.softmax(logits, -1)
    z = s + a["gate_bias"].double() if a["gate_bias"] is not None else s.clone()
    gaps = [torch.full((T,), math.inf, dtype=torch.float64, device="cuda")]
    if G > 1:
        zg = z.view(T, G, E // G)
        best, order = zg.topk(2 if a["gate_bias"] is not None else 1, -1)[0].sum(-1).sort(dim=-1, descending=True)
        if TG < G:
            gaps.append(best[:, TG - 1] - best[:, TG])
        keep = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, order[:, :TG], True)
        z = zg.masked_fill(~keep[..., None], -math.inf).reshape(T, E)
    v, order = z.sort(dim=-1, descending=True)
    gaps.append((v[:, :topk] - v[:, 1:topk + 1]).amin(-1) if topk < E else (v[:, :-1] - v[:, 1:]).amin(-1))
    idx = order[:, :topk]
    w = s.gather(1, idx)
    w = (w / w.sum(-1, keepdim=True) if normalize else w) * scale
    return idx, w, torch.stack(gaps).amin(0)


def run_layer(a, topk, ns, G=1, TG=1, score=fb.SCORE_SIGMOID, scale=1.0, normalize=True, ue8m0=False, **kw):
    return fb.moe_layer(a["x"], a["gate_w"], a["w1"], a["w1_s"], a["w3"], a["w3_s"], a["w2"], a["w2_s"], topk=topk,
                        gate_bias=a["gate_bias"], n_groups=G, topk_groups=TG, score_func=score, route_scale=scale,
                        normalize=normalize, n_shared=ns, scale_fmt=fb.SCALE_UE8M0 if ue8m0 else fb.SCALE_FP32, **kw)


CASES = [
    # T, dim, inter, E, topk, shared, groups, kept, sigmoid, bias, ue8m0
    (1, 128, 128, 32, 1, 0, 1, 1, True, False, False),
    (1, 512, 256, 64, 6, 2, 1, 1, False, False, False),
    (2, 1024, 384, 32, 4, 1, 4, 2, True, True, True),
    (7, 640, 128, 96, 8, 0, 8, 3, False, True, False),
    (8, 2048, 1408, 64, 6, 2, 1, 1, False, False, False),
    (9, 768, 640, 160, 6, 2, 8, 3, False, False, False),
    (16, 1280, 256, 256, 8, 1, 8, 4, True, True, True),
    (17, 384, 512, 32, 32, 1, 1, 1, True, True, False),
    (24, 896, 384, 64, 2, 8, 2, 1, True, False, False),
    (31, 1664, 896, 128, 8, 1, 4, 4, True, True, False),
    (32, 512, 128, 32, 3, 0, 32, 5, False, False, True),
    (3, 7168, 2048, 32, 8, 1, 8, 4, True, True, False),
    (4, 8192, 2176, 32, 2, 0, 1, 1, True, False, False),
    (32, 4096, 2304, 32, 6, 1, 1, 1, False, False, False),
]


@pytest.mark.parametrize("T,dim,inter,E,topk,ns,G,TG,sig,bias,ue8m0", CASES)
def test_layer(T, dim, inter, E, topk, ns, G, TG, sig, bias, ue8m0):
    a = make(T, dim, inter, E, ns, 50 + T + dim, bias, ue8m0)
    score = fb.SCORE_SIGMOID if sig else fb.SCORE_SOFTMAX
    normalize = T % 2 == 0
    idx = torch.full((T, topk), -7, dtype=torch.int32, device="cuda")
    w = torch.zeros((T, topk), device="cuda")
    kw = dict(G=G, TG=TG, score=score, scale=1.5, normalize=normalize, ue8m0=ue8m0)
    y = run_layer(a, topk, ns, idx=idx, w=w, **kw)
    torch.cuda.synchronize()
    assert fb.last_device_error() == 0
    ids, wr, gap = routing(a, topk, G, TG, score, 1.5, normalize)
    sure = gap > 1e-6 * (1 if sig else 1 / 32)   # fp32 scores: no choice closer than their error
    assert sure.double().mean() >= 0.9
    assert torch.equal(idx.long()[sure], ids[sure])
    assert ((w.double() - wr)[sure].abs() <= 2e-5 * wr[sure]).all()
    ref, tol = reference(a, idx.long(), w, ns, ue8m0)
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert float(err.norm() / ref.norm()) <= 3e-3, float(err.norm() / ref.norm())
    again = run_layer(a, topk, ns, **kw)
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


def test_layer_ties_go_to_the_lower_expert():
    """Equal gate rows give equal logits: the lower ids are taken."""
    a = make(5, 256, 128, 64, 0, 1)
    a["gate_w"][:] = a["gate_w"][:1]
    idx = torch.empty((5, 4), dtype=torch.int32, device="cuda")
    run_layer(a, 4, 0, idx=idx)
    assert torch.equal(idx, torch.arange(4, dtype=torch.int32, device="cuda").expand(5, 4))


def test_layer_all_tokens_on_the_same_experts_and_zero_rows():
    """One expert set for every token (the fullest column tiles); a zero token
    gives a zero row."""
    a = make(32, 512, 256, 64, 1, 2)
    a["x"][:] = a["x"][:1]
    a["x"][13] = 0
    idx = torch.empty((32, 8), dtype=torch.int32, device="cuda")
    w = torch.empty((32, 8), device="cuda")
    y = run_layer(a, 8, 1, idx=idx, w=w)
    rest = [t for t in range(32) if t != 13]
    assert (y[13] == 0).all() and torch.equal(y[rest], y[:1].expand(31, 512))
    ref, tol = reference(a, idx.long(), w, 1, False)
    assert ((y.double() - ref).abs() <= tol).all()


def test_layer_agrees_with_the_chained_kernels():
    """Against act_quant, moe_gate and moe_grouped_gemm, which round their
    intermediates to bf16: h1, h3, silu and u (each 1.66e-3 rms of the value, so
    u within 3.4e-3, and the quantisation of u takes another code where that
    crosses a border: a code step of 2^-3 with probability about 2 * 3.4e-3 /
    2^-3, an rms of 2^-3 sqrt(0.054 / 3) = 1.7e-2), then outputs and sums. 2.5e-2
    of the output's norm covers them."""
    T, dim, inter, E, ns, k = 12, 1024, 512, 64, 1, 6
    a = make(T, dim, inter, E, ns, 3, bias=True)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    y = run_layer(a, k, ns, idx=idx, w=w)
    q, s = fb.act_quant(a["x"])
    z = fb.moe_grouped_gemm(q, s, idx, w, a["w1"], a["w1_s"], a["w3"], a["w3_s"], a["w2"], a["w2_s"], E, n_shared=ns)
    assert float((y.double() - z.double()).norm() / y.double().norm()) <= 2.5e-2


def test_layer_workspace_is_left_ready_and_shared_by_shapes():
    """Calls of different shapes in a row on one workspace, zeroed once."""
    shapes = [(1, 512, 256, 64, 6, 2), (32, 1024, 384, 32, 4, 1), (9, 256, 128, 256, 8, 0), (1, 512, 256, 64, 6, 2)]
    n = max(fb.moe_layer_workspace_bytes(T, k, E, d, i, ns) for T, d, i, E, k, ns in shapes)
    buf = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = buf[(-buf.data_ptr()) % 256:][:n]
    ws[:256] = 0
    args = [(make(T, d, i, E, ns, 60 + T), k, ns) for T, d, i, E, k, ns in shapes]
    got = [run_layer(a, k, ns, ws=ws) for a, k, ns in args]
    torch.cuda.synchronize()
    assert (ws[:256] == 0).all()
    for (a, k, ns), y in zip(args, got):
        assert torch.equal(run_layer(a, k, ns).view(torch.int16), y.view(torch.int16))
    with pytest.raises(fb.Fp8BlkError):
        run_layer(args[1][0], 4, 1, ws=ws[:fb.moe_layer_workspace_bytes(32, 4, 32, 1024, 384, 1) - 1])
    assert fb.last_device_error() == 0


def test_layer_leaves_every_counter_at_zero():
    """Also those of row tiles that this shape does not have (512 rows: the first 4 of 64), where another shape's call
    that gave up may have left a part of a count."""
    a = make(3, 512, 256, 64, 1, 8)
    ref = run_layer(a, 6, 1)
    buf = torch.zeros(fb.moe_layer_workspace_bytes(3, 6, 64, 512, 256, 1) + 256, dtype=torch.uint8, device="cuda")
    ws = buf[(-buf.data_ptr()) % 256:]
    ws[64 + 4:64 + 64] = 0x11      # row tile k's count is byte 64 + k
    y = run_layer(a, 6, 1, ws=ws)
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
    assert (ws[:256] == 0).all() and fb.last_device_error() == 0


def test_layer_in_a_graph_and_on_a_side_stream():
    a = make(4, 512, 256, 64, 1, 5)
    ref = run_layer(a, 6, 1)
    out = torch.empty_like(ref)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run_layer(a, 6, 1, out=out)
        stream.synchronize()
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run_layer(a, 6, 1, out=out)
    x2 = a["x"].flip(0).contiguous()
    a["x"].copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), ref.flip(0).contiguous().view(torch.int16))


def test_layer_refusals():
    a = make(4, 512, 256, 64, 1, 6)
    assert run_layer(a | dict(x=a["x"][:0]), 6, 1).shape == (0, 512)
    big = make(33, 128, 128, 32, 0, 7)
    with pytest.raises(fb.Fp8BlkError):
        run_layer(big, 2, 0)
    for bad in (dict(x=a["x"].float()), dict(x=a["x"][:, :384]), dict(gate_w=a["gate_w"][:63]),
                dict(w1=a["w1"][:-1]), dict(w2_s=a["w2_s"][:-1]), dict(w3_s=a["w3_s"].double()),
                dict(gate_bias=torch.zeros(63, device="cuda")), dict(x=a["x"].cpu()), dict(x=a["x"].t())):
        with pytest.raises(fb.Fp8BlkError):
            run_layer(a | bad, 6, 1)
    for kw in (dict(topk=0), dict(topk=33), dict(G=3), dict(G=4, TG=5), dict(score=2), dict(scale=math.nan),
               dict(topk=20, G=8, TG=2), dict(ns=2)):
        args = dict(topk=6, ns=1) | kw
        with pytest.raises(fb.Fp8BlkError):
            run_layer(a, **args)
    assert fb.moe_layer_workspace_bytes(33, 6, 64, 512, 256) == 0
    assert fb.last_device_error() == 0
