"""The norm around a block against 64 bits.

Tolerances. A sum of D squares in fp32 (16 in a thread, then lanes, then warps) is off by at most (16 + 10) 2^-24 of
itself, its root by half of that, and a value passes at most eight more roundings: 2^-19 relative for z, and 2^-19 (|gate z| + |rs x|)
for r before it is rounded. With q = |gate z| + |rs x|, the norm of r moves by at most 2^-19 sqrt(sum q^2 / sum r^2)
relative, so h before its rounding is off by E = 2^-19 (q / rms(r) |w| + |h| (1 + sqrt(sum q^2 / sum r^2))). The roundings
add half a step each: 2^-8 of the value in bf16; quantised outputs are held to the codes and scales that the rules give
between h - E and h + E."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(T, D, seed, post, gate, x=True, strided=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s, std=1.0):
        return torch.randn(*s, generator=g, device="cuda") * std

    pad = 64 if strided else 0
    return {"y": normal(T, D + pad).bfloat16()[:, pad:], "x": normal(T, D + pad, std=3.0).bfloat16()[:, :D] if x else None,
            "norm_w": 1 + normal(D, std=0.2), "post_w": 0.5 + normal(D, std=0.2) if post else None,
            "gate": {None: None, "column": 1 + normal(D, std=0.3), "token": normal(T, D + pad).bfloat16()[:, pad:]}[gate]}


def formula(a, rs, eps=EPS):
    """r, h and E in 64 bits."""
    z = a["y"].double()
    if a["post_w"] is not None:
        z = z / (z.pow(2).mean(-1, keepdim=True) + eps).sqrt() * a["post_w"].double()
    if a["gate"] is not None:
        z = z * a["gate"].double()
    x = a["x"].double() * rs if a["x"] is not None else torch.zeros_like(z)
    r, q = x + z, x.abs() + z.abs()
    rms = (r.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    h = r / rms * a["norm_w"].double()
    ratio = (q.pow(2).sum(-1, keepdim=True) / r.pow(2).sum(-1, keepdim=True).clamp(min=1e-300)).sqrt()
    E = 2.0 ** -19 * (q / rms * a["norm_w"].double().abs() + h.abs() * (1 + ratio))
    return r, 2.0 ** -19 * q, h, E


def close(got, want, slack):
    off = (got.double() - want).abs()
    # (2^-134: half of the smallest bf16 step)
    bad = ~(off <= 2.0 ** -8 * want.abs() + slack * (1 + 2.0 ** -7) + 2.0 ** -134)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


CASES = [(1, 7168, False, None, 1.0), (3, 5120, True, "column", 1.0), (130, 2048, True, "token", 0.5),
         (17, 1536, False, "token", 1.4), (5, 128, True, "column", -0.7), (2, 16384, True, "token", 1.0),
         (300, 8320, False, "column", 1.0), (9, 8192, True, None, 1.0), (1025, 512, True, None, 1.0), (4, 384, False, None, 0.0)]


@pytest.mark.parametrize("T,D,post,gate,rs", CASES + [(1, 8, True, "token", 1.0), (4, 24, False, "column", 2.0),
                                                      (6, 1000, True, "token", 1.0), (2, 8200, True, "column", 1.0),
                                                      (33, 4808, False, "token", 1.0)])
@pytest.mark.parametrize("strided", [False, True])
def test_bf16(T, D, post, gate, rs, strided):
    a = make(T, D, T + D, post, gate, strided=strided)
    r, h = fb.residual_norm(**a, residual_scale=rs, eps=EPS)
    wr, er, wh, eh = formula(a, rs)
    close(r, wr, er)
    close(h, wh, eh)


@pytest.mark.parametrize("D", [8, 512, 7168])
def test_without_a_residual(D):
    a = make(3, D, 1, False, None, x=False)
    r, h = fb.residual_norm(**a, eps=EPS)
    assert torch.equal(r, a["y"])
    wr, er, wh, eh = formula(a, 1.0)
    close(h, wh, eh)


@pytest.mark.parametrize("T,D,post,gate,rs", CASES)
@pytest.mark.parametrize("ue8m0", [False, True])
def test_fp8(T, D, post, gate, rs, ue8m0):
    a = make(T, D, T + D + 1, post, gate)
    r, (q, s) = fb.residual_norm(**a, residual_scale=rs, eps=EPS, quant="fp8",
                                 scale_fmt=fb.SCALE_UE8M0 if ue8m0 else fb.SCALE_FP32)
    wr, er, wh, eh = formula(a, rs)
    close(r, wr, er)
    lo, hi = wh - eh, wh + eh

    def scale(sign):      # of the block's largest |h|, one more fp32 rounding below or above
        m = (wh.abs() + sign * eh).clamp(min=0).view(T, -1, 128).amax(-1).clamp(min=1e-4) / 448 * (1 + sign * 2.0 ** -22)
        return torch.exp2(torch.ceil(torch.log2(m))) if ue8m0 else m

    assert q.dtype is torch.float8_e4m3fn and s.shape == (T, D // 128)
    assert bool(((s >= scale(-1)) & (s <= scale(1))).all())
    sd = s.double().repeat_interleave(128, 1)
    code = lambda v: (v / sd).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()  # noqa: E731
    got, d = q.double(), 2.0 ** -22      # the quotient's own rounding, and .float()'s here
    assert bool(((got >= code(lo - d * lo.abs())) & (got <= code(hi + d * hi.abs()))).all())


@pytest.mark.parametrize("T,D,post,gate,rs", CASES)
@pytest.mark.parametrize("fmt", [fb.FP4_E4M3, fb.FP4_UE8M0])
def test_fp4(T, D, post, gate, rs, fmt):
    a = make(T, D, T + D + 2, post, gate)
    r, (q, s, g) = fb.residual_norm(**a, residual_scale=rs, eps=EPS, quant="fp4", scale_fmt=fmt)
    wr, er, wh, eh = formula(a, rs)
    close(r, wr, er)
    wh, eh = wh.cpu().numpy(), eh.cpu().numpy()
    s = ref.untiled(s.cpu().numpy(), T)
    per = 16 if fmt == fb.FP4_E4M3 else 32
    blocks = lambda v: v.reshape(T, -1, per).max(-1)  # noqa: E731
    d = 2.0 ** -21      # the rule's own fp32 roundings
    big, small = (np.abs(wh) + eh) * (1 + d), np.maximum(np.abs(wh) - eh, 0) * (1 - d)
    if fmt == fb.FP4_E4M3:
        g = g.cpu().numpy().astype(np.float64)
        assert np.all((g >= small.max(-1) / 2688 * (1 - d)) & (g <= big.max(-1) / 2688 * (1 + d)))
        bound = lambda v, top: ref.nearest(blocks(v) * (448 / top)[:, None], ref.E4M3_VALUES)  # noqa: E731
        assert np.all((s >= bound(small, big.max(-1))) & (s <= bound(big, small.max(-1))))
        unit = ref.E4M3_VALUES[s] * g[:, None]
    else:
        assert g is None
        bound = lambda v: np.maximum(np.ceil(np.log2(np.maximum(blocks(v) / 6, 2.0 ** -140))), -126) + 127  # noqa: E731
        assert np.all((s >= bound(small)) & (s <= bound(big)))
        unit = np.ldexp(1.0, s.astype(np.int64) - 127)
    unit = unit.repeat(per, 1)
    with np.errstate(all="ignore"):
        at = lambda v: np.where(unit > 0, ref.VALUES[ref.nearest(np.abs(v / unit), ref.VALUES)] * np.sign(v), 0)  # noqa: E731
        codes = ref.unpack(q.cpu().numpy())
        got = ref.VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
        lo, hi = wh - eh - d * np.abs(wh), wh + eh + d * np.abs(wh)
        assert np.all((got >= at(lo)) & (got <= at(hi)))


@pytest.mark.parametrize("quant", [None, "fp8", "fp4"])
def test_in_place(quant):
    """r may take the place of x, or of y."""
    for name in ("x", "y"):
        a = make(67, 1536, 8, True, "column")
        want = fb.residual_norm(**a, quant=quant)
        got = fb.residual_norm(**a, quant=quant, r=a[name])
        assert got[0].data_ptr() == a[name].data_ptr() and torch.equal(got[0], want[0])
        for u, v in zip(got[1] if quant else got[1:], want[1] if quant else want[1:]):
            if u is not None and u.dim() < 5:      # (scale tiles also hold bytes of rows that are not there)
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_edges():
    """A row of zeros stays zeros; a row with a NaN or an infinity is its own affair; tiny and huge rows."""
    D = 256
    a = make(6, D, 3, False, None, x=False)
    a["y"][0] = 0
    a["y"][1, 7] = float("nan")
    a["y"][2, 9] = float("inf")
    a["y"][3] *= 2.0 ** -120
    a["y"][4] *= 2.0 ** 60
    a["y"][5] = 0
    r, h = fb.residual_norm(**a)
    assert torch.equal(r.isnan(), a["y"].isnan())
    assert bool((h[0] == 0).all()) and bool(h[1].isnan().all()) and bool(h[2, 9].isnan()) and not bool(h[3:].isnan().any())
    wr, er, wh, eh = formula({**a, "y": a["y"][4:5]}, 1.0)
    close(h[4:5], wh, eh)
    for fmt in (fb.FP4_E4M3, fb.FP4_UE8M0):
        _, (q, s, g) = fb.residual_norm(**a, quant="fp4", scale_fmt=fmt)
        d = fb.fp4_dequant(q, s, g, fmt)
        assert bool((d[0] == 0).all()) and bool(d[1].isnan().all()) and bool(d[2].isnan().any())
        assert not bool(d[3:].isnan().any())


def test_refusals():
    a = make(4, 256, 3, False, None)
    y = a["y"]
    tok = torch.ones(4, 256, device="cuda").bfloat16()
    bad = [
        lambda: fb.residual_norm(y.float(), y, a["norm_w"]), lambda: fb.residual_norm(y, y[:3], a["norm_w"]),
        lambda: fb.residual_norm(y, y, a["norm_w"].bfloat16()), lambda: fb.residual_norm(y, y, a["norm_w"][:128]),
        lambda: fb.residual_norm(y, y, a["norm_w"], post_w=a["norm_w"][:128]),
        lambda: fb.residual_norm(y, y, a["norm_w"], gate=tok[:3]), lambda: fb.residual_norm(y, y, a["norm_w"], gate=tok.float()),
        lambda: fb.residual_norm(y, y, a["norm_w"], gate=tok[:, 0]), lambda: fb.residual_norm(y, y, a["norm_w"], quant="int8"),
        lambda: fb.residual_norm(y[:, :120], None, a["norm_w"][:120], quant="fp8"),
        lambda: fb.residual_norm(y, y, a["norm_w"], quant="fp4", scale_fmt=9), lambda: fb.residual_norm(y, y, a["norm_w"], eps=-1.0),
        lambda: fb.residual_norm(y.t(), y.t(), a["norm_w"]), lambda: fb.residual_norm(y, y, a["norm_w"], r=tok[:, :128]),
        lambda: fb.residual_norm(torch.zeros(2, 16392, device="cuda").bfloat16(), None, torch.ones(16392, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(fb.Fp8BlkError):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("fmt", [fb.FP4_E4M3, fb.FP4_UE8M0])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_the_seam_feeds_the_products(T, fmt):
    """Norm, product, norm, product as a layer runs them, without and with a graph: the same numbers as call by call."""
    D, N = 1024, 1536
    a = make(T, D, 5, True, "column")
    g = torch.Generator(device="cuda").manual_seed(6)
    up = fb.fp4_quant(torch.randn(N, D, generator=g, device="cuda") * D ** -0.5, fmt)
    down = fb.weight_quant(torch.randn(D, N, generator=g, device="cuda") * N ** -0.5)
    w2 = 1 + torch.randn(N, generator=g, device="cuda") * 0.1
    torch.cuda.synchronize()

    def layer(sync=lambda: None):
        r, h = fb.residual_norm(**a, quant="fp4", scale_fmt=fmt)
        sync()
        u = fb.fp4_gemm(*h, *up, fmt)
        sync()
        _, (q, s) = fb.residual_norm(u, None, w2, quant="fp8")
        sync()
        y = fb.fp8_gemm(q, s, *down)
        sync()
        return fb.residual_norm(y, r, a["norm_w"], residual_scale=0.5)

    want = layer(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(layer(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = layer()
    y0 = a["y"].clone()
    a["y"].zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got[0], want[0])
    a["y"].copy_(y0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    assert fb.last_device_error() == 0
