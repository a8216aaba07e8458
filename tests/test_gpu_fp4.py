"""Microscaled 4-bit floats: quantisation bit for bit, products against 64 bits.

Tolerance of a product: bf16 rounds once, by at most half a step (2^-8 of the value); the tensor cores sum 64 columns at
a time into fp32, each step off by at most 2^-21 of the sum of the products' sizes S (truncation and alignment within the
64 products), the two row scales by 2^-23: |c - ref| <= 2^-8 |ref| + (K / 64 + 2) 2^-21 S."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu
FORMATS = [fb.FP4_E4M3, fb.FP4_UE8M0]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def random_rows(M, K, seed):
    """bf16 values (as float32) whose blocks differ in size by many powers of two."""
    r = np.random.RandomState(seed)
    x = r.randn(M, K) * np.exp2(r.randint(-12, 6, size=(M, K // 32))).repeat(32, 1)
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def check_quant(x, fmt, got):
    q, s, g = got
    codes, sb, row = ref.quant(x.float().cpu().numpy(), fmt)
    M, K = codes.shape
    assert tuple(s.shape) == fb.fp4_scale_shape(M, K, fmt)
    assert np.array_equal(ref.untiled(s.cpu().numpy(), M), sb)
    if fmt == fb.FP4_E4M3:
        assert np.array_equal(g.cpu().numpy(), row, equal_nan=True)
    else:
        assert g is None
    assert np.array_equal(ref.unpack(q.cpu().numpy()), codes)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (33, 384), (129, 1536), (200, 2048), (7, 7168), (2, 16384), (5, 18432),
                                 (1, 40064)])
def test_quant_is_the_rule(M, K, fmt):
    x = random_rows(M, K, M + K).cuda()
    check_quant(x, fmt, fb.fp4_quant(x, fmt))
    x = (x.float() * 1.2345).contiguous()      # fp32 that is no bf16
    check_quant(x, fmt, fb.fp4_quant(x, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quant_of_strided_rows(fmt):
    x = random_rows(37, 1024, 1).cuda()
    check_quant(x[:, 256:768], fmt, fb.fp4_quant(x[:, 256:768], fmt))
    check_quant(x[::3], fmt, fb.fp4_quant(x[::3], fmt))


def edge_rows():
    """Rows whose values sit where a rule turns: zeros, signed zeros, subnormals, the largest numbers, ties, one large
    value among small ones, NaN and infinities."""
    K = 256
    rows = []
    rows.append(np.zeros(K))
    rows.append(np.where(np.arange(K) % 2, -0.0, 0.0))
    rows.append(np.full(K, 2.0 ** -133))
    rows.append(np.full(K, 2.0 ** -126))
    rows.append(np.where(np.arange(K) % 3, 3.3e38, -2.0 ** 127))
    rows.append(np.concatenate([ref.MID, -ref.MID, ref.VALUES, -ref.VALUES, [5.0, 6.0]]).repeat(8)[:K])   # ties at s = 1
    rows.append(np.where(np.arange(K) == 77, 1e6, 1e-3))
    rows.append(np.where(np.arange(K) == 77, np.nan, 1.0))
    rows.append(np.where(np.arange(K) == 177, np.inf, 1.0))
    rows.append(np.where(np.arange(K) == 9, -np.inf, 0.0))
    rows.append(2.0 ** (np.arange(K) % 40 - 20.0))
    x = np.stack([np.resize(r, K) for r in rows]).astype(np.float32)
    return x


@pytest.mark.parametrize("fmt", FORMATS)
def test_quant_edges(fmt):
    x = dev(edge_rows())
    check_quant(x, fmt, fb.fp4_quant(x, fmt))
    b = x.bfloat16()
    check_quant(b, fmt, fb.fp4_quant(b, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 128), (130, 384), (257, 2048)])
def test_dequant(M, K, fmt):
    """One fp32 multiply, one rounding: half a bf16 step and half an fp32 step from q s g."""
    r = np.random.RandomState(M)
    codes = r.randint(0, 16, (M, K)).astype(np.uint8)
    if fmt == fb.FP4_E4M3:
        s, g = r.randint(0, 0x7F, (M, K // 16)).astype(np.uint8), np.exp(r.randn(M)).astype(np.float32)
    else:
        s, g = r.randint(0, 240, (M, K // 32)).astype(np.uint8), None
        s[0, 0], s[-1, -1] = 0, 255
    out = fb.fp4_dequant(dev(ref.pack(codes)), dev(ref.tiles(s)), None if g is None else dev(g), fmt)
    want = ref.values(codes, s, g, fmt)
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    off = np.abs(got - want)[fine]
    # below the smallest normal bf16 a step is 2^-133
    assert np.all(off <= np.abs(want[fine]) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -134)


def operands(M, N, K, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, K, generator=g, device="cuda") * 0.05
    return quantised(a, w, fmt)


def quantised(a, w, fmt):
    """Both operands, finished: a weight may be read before the calls just before the product have ended."""
    both = fb.fp4_quant(a, fmt), fb.fp4_quant(w, fmt)
    torch.cuda.synchronize()
    return both


def dense(op, fmt):
    q, s, g = op
    codes = ref.unpack(q.cpu().numpy())
    v = ref.values(codes, ref.untiled(s.cpu().numpy(), codes.shape[0]), None if g is None else g.cpu().numpy(), fmt)
    return torch.from_numpy(v).cuda()


def check_product(c, a, w, K):
    want = a @ w.t()
    size = a.abs() @ w.abs().t()
    off = (c.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (K // 64 + 2) * 2.0 ** -21 * size
    bad = off > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:4].tolist()}: " \
                          f"{c[bad][:4].tolist()} for {want[bad][:4].tolist()}"


SHAPES = [(1, 1, 128), (1, 128, 256), (1, 2112, 7168), (2, 129, 384), (7, 576, 2048), (16, 1000, 1536), (17, 257, 640),
          (32, 2048, 512), (33, 500, 1280), (64, 1536, 2048), (65, 384, 2176), (100, 7, 896), (128, 512, 1024),
          (129, 300, 768), (255, 640, 384), (300, 1000, 1152), (513, 777, 2048), (1025, 520, 256), (8, 24576, 1536),
          (640, 5120, 512), (770, 2568, 1408), (2049, 1030, 640), (1, 64, 18432), (260, 264, 18432)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, fmt):
    a, w = operands(M, N, K, fmt, M * 7 + N)
    c = fb.fp4_gemm(*a, *w, fmt)
    check_product(c, dense(a, fmt), dense(w, fmt), K)
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [9, 200, 1200])
def test_gemm_keeps_its_neighbours(M, fmt):
    """The bytes before and after the output stay as they were, for outputs at odd places too."""
    N, K = 333, 512
    a, w = operands(M, N, K, fmt, 5)
    want = fb.fp4_gemm(*a, *w, fmt)
    for shift in (1, 8):
        buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[shift:shift + M * N].view(M, N)
        fb.fp4_gemm(*a, *w, fmt, out=out)
        assert torch.equal(out, want)
        assert bool((buf[:shift] == 7).all()) and bool((buf[shift + M * N:] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [3, 150, 700])
def test_gemm_keeps_bad_rows_apart(M, fmt):
    """A token with a NaN or an infinity is NaN in its row alone, a weight row in its column; what the scale bytes
    behind the last row hold does not matter."""
    N, K = 300, 640
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    wt = torch.randn(N, K, generator=g, device="cuda")
    x[1, 5], wt[17, 600] = float("inf"), float("nan")
    a, w = quantised(x, wt, fmt)
    for op, rows in ((a, M), (w, N)):
        flat = op[1].permute(0, 3, 2, 1, 4).reshape(-1, op[1].shape[1] * 4)      # a copy [rows, blocks]
        flat[rows:] = 255
        op[1].copy_(flat.view(op[1].shape[0], 4, 32, op[1].shape[1], 4).permute(0, 3, 2, 1, 4))
    c = fb.fp4_gemm(*a, *w, fmt)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[1], bad[:, 17] = True, True
    assert torch.equal(c.isnan(), bad)
    da, dw = dense(a, fmt).nan_to_num(0.0), dense(w, fmt).nan_to_num(0.0)
    check_product(torch.where(bad, (da @ dw.t()).bfloat16(), c), da, dw, K)


@pytest.mark.parametrize("fmt", FORMATS)
def test_gemm_large_and_small_numbers(fmt):
    """Row scales (E4M3) or block scales (UE8M0) at both ends of their range: products stay within bf16's."""
    M, N, K = 40, 200, 256
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(M, K, generator=g, device="cuda") * torch.exp2(torch.linspace(-60, 60, M, device="cuda"))[:, None]
    wt = torch.randn(N, K, generator=g, device="cuda") * torch.exp2(torch.linspace(-50, 50, N, device="cuda"))[:, None]
    a, w = quantised(x.bfloat16(), wt, fmt)
    check_product(fb.fp4_gemm(*a, *w, fmt), dense(a, fmt), dense(w, fmt), K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 640, 1536), (8, 10944, 2048), (150, 333, 384), (1024, 1536, 7168)])
def test_linear_is_quant_and_gemm(M, N, K, fmt):
    x = random_rows(M, K + 64, 9).cuda()[:, 64:]
    _, w = operands(1, N, K, fmt, 11)
    want = fb.fp4_gemm(*fb.fp4_quant(x, fmt), *w, fmt)
    assert torch.equal(fb.fp4_linear(x, *w, fmt), want)
    nb = fb.fp4_linear_workspace_bytes(M, N, K, fmt)
    ws = torch.full((nb + 256,), 171, dtype=torch.uint8, device="cuda")
    off = -ws.data_ptr() % 256
    assert torch.equal(fb.fp4_linear(x, *w, fmt, ws=ws[off:off + nb]), want)
    assert bool((ws[off + nb:] == 171).all()) and bool((ws[:off] == 171).all())


def test_empty_sizes():
    _, w = operands(1, 64, 256, fb.FP4_E4M3, 0)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    assert fb.fp4_linear(x, *w).shape == (0, 64)
    q, s, g = fb.fp4_quant(x)
    assert q.shape == (0, 128) and s.shape == (0, 4, 32, 4, 4) and g.shape == (0,)
    assert fb.fp4_dequant(q, s, g).shape == (0, 256)
    assert fb.fp4_gemm(q, s, g, *w).shape == (0, 64)
    a = fb.fp4_quant(torch.randn(5, 256, device="cuda"))
    assert fb.fp4_gemm(*a, q, s, g).shape == (5, 0)
    z = lambda n: (torch.empty(n, 0, dtype=torch.uint8, device="cuda"),  # noqa: E731
                   torch.empty(fb.fp4_scale_shape(n, 0), dtype=torch.uint8, device="cuda"), torch.ones(n, device="cuda"))
    out = torch.full((3, 4), 9.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fb.fp4_gemm(*z(3), *z(4), out=out), torch.zeros_like(out))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [4, 600])
def test_calls_in_a_row_and_in_a_graph(M, fmt):
    """Layers of different shapes back to back, each reading what the one before wrote, on a stream of their own, then
    captured and replayed on new inputs."""
    dims = [512, 1408, 384, 2048, 512]
    ws = [operands(1, n, k, fmt, n)[1] for k, n in zip(dims, dims[1:])]

    def chain(x):
        for w in ws:
            x = fb.fp4_linear(x, *w, fmt)
        return x

    def stepwise(x):
        for w in ws:
            q = fb.fp4_quant(x, fmt)
            torch.cuda.synchronize()
            x = fb.fp4_gemm(*q, *w, fmt)
            torch.cuda.synchronize()
        return x

    xs = [torch.randn(M, 512, device="cuda").bfloat16() for _ in range(3)]
    want = [stepwise(x) for x in xs]
    assert torch.equal(chain(xs[0]), want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = xs[1].clone()
        assert torch.equal(chain(x), want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = chain(x)
    torch.cuda.synchronize()
    for i in (2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    assert fb.last_device_error() == 0


def test_results_do_not_vary():
    a, w = operands(24, 2112, 7168, fb.FP4_E4M3, 2)
    first = fb.fp4_gemm(*a, *w)
    for _ in range(20):
        assert torch.equal(fb.fp4_gemm(*a, *w), first)


def test_refusals():
    a, w = operands(4, 64, 256, fb.FP4_E4M3, 1)
    x = torch.randn(4, 256, device="cuda").bfloat16()
    bad = [
        lambda: fb.fp4_quant(x.half()), lambda: fb.fp4_quant(x[:, :200]), lambda: fb.fp4_quant(x.t()),
        lambda: fb.fp4_quant(x, 2), lambda: fb.fp4_quant(x.cpu()), lambda: fb.fp4_quant(x[None]),
        lambda: fb.fp4_quant(torch.randn(4, 260, device="cuda").bfloat16()[:, 1:129]),        # misaligned
        lambda: fb.fp4_quant(torch.randn(4, 257, device="cuda").bfloat16()[:, :256]),         # stride
        lambda: fb.fp4_gemm(a[0], a[1], None, *w), lambda: fb.fp4_gemm(a[0][:, :64].contiguous(), a[1], a[2], *w),
        lambda: fb.fp4_gemm(*a, w[0], w[1], w[2][:63]), lambda: fb.fp4_gemm(*a, w[0], w[1][:, :1], w[2]),
        lambda: fb.fp4_gemm(*a, *w, fb.FP4_UE8M0), lambda: fb.fp4_gemm(*a, *w, out=x),
        lambda: fb.fp4_gemm(*a, *w, out=torch.empty(4, 64, device="cuda")),
        lambda: fb.fp4_linear(x[:, :128], *w), lambda: fb.fp4_linear(x.float(), *w),
        lambda: fb.fp4_linear(x, *w, ws=torch.empty(256, dtype=torch.uint8, device="cuda")),
        lambda: fb.fp4_dequant(a[0], a[1], a[2][:3]), lambda: fb.fp4_dequant(a[0].int(), a[1], a[2]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(fb.Fp8BlkError):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(3, 300, 640), (1, 2112, 7168), (5, 128, 1536)])
def test_linear_keeps_bad_tokens_apart(M, N, K, fmt):
    """Few tokens are quantised by the product's own blocks: zeros, a NaN, an infinity and far scales as by fp4_quant."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(M, K, generator=g, device="cuda")
    _, w = quantised(x, torch.randn(N, K, generator=g, device="cuda"), fmt)
    bad = []
    for i, what in enumerate(["zero", "nan", "inf", "small", "large"]):
        y = x.clone()
        row = i % M
        if what == "zero":
            y[row] = 0
        elif what == "nan":
            y[row, K // 2] = float("nan")
        elif what == "inf":
            y[row, 3] = -float("inf")
        else:
            y[row] *= 2.0 ** (-110 if what == "small" else 100)
        y = y.bfloat16()
        got, want = fb.fp4_linear(y, *w, fmt), fb.fp4_gemm(*fb.fp4_quant(y, fmt), *w, fmt)
        if not (torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))):
            bad.append(what)
        if what in ("nan", "inf"):
            assert bool(got[row].isnan().all()) and int(got.isnan().any(1).sum()) == 1
    assert not bad


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 8192), (1, 8320), (2, 2048), (2, 2176), (16, 256), (16, 384), (17, 256)])
def test_linear_on_both_sides_of_the_fused_sizes(M, K, fmt):
    """Where the activations stop being quantised inside the product, the numbers stay the same."""
    x = random_rows(M, K, M * K).cuda()
    _, w = operands(1, 333, K, fmt, 5)
    want = fb.fp4_gemm(*fb.fp4_quant(x, fmt), *w, fmt)
    assert torch.equal(fb.fp4_linear(x, *w, fmt), want)


def test_two_streams():
    """Products split over clusters, of pairs, and an FP8 linear, from two streams at once: they
    share SMs (and columns of tensor memory), and each gives what it gives alone."""
    fmt = fb.FP4_E4M3
    shapes = [(8, 2112, 7168), (100, 1533, 1536), (1, 2112, 7168), (40, 640, 7168), (100, 333, 7168), (600, 1536, 512)]
    pairs = [operands(m, n, k, fmt, i) for i, (m, n, k) in enumerate(shapes)]
    x8 = torch.randn(4, 2048, device="cuda").bfloat16()
    w8 = fb.weight_quant(torch.randn(1408, 2048, device="cuda"))
    torch.cuda.synchronize()
    want = [fb.fp4_gemm(*a, *w, fmt) for a, w in pairs]
    want8 = fb.linear(x8, *w8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(12):
        for side, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                for i in range(len(pairs)):
                    j = (i + turn + 3 * side) % len(pairs)
                    got[side].append((want[j], fb.fp4_gemm(*pairs[j][0], *pairs[j][1], fmt)))
                got[side].append((want8, fb.linear(x8, *w8)))
    torch.cuda.synchronize()
    for side in got:
        for a, b in side:
            assert torch.equal(a, b)
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1024, 7168, 2048), (700, 7168, 2432), (600, 7000, 2176), (1000, 7272, 2560), (2000, 3400, 2176),
                                   (769, 6920, 2176)])
def test_gemm_by_wide_tiles(M, N, K, fmt):
    """Products whose tiles go a round less where they are wider, with last tiles of every width."""
    a, w = operands(M, N, K, fmt, M + N)
    check_product(fb.fp4_gemm(*a, *w, fmt), dense(a, fmt), dense(w, fmt), K)
    assert fb.last_device_error() == 0
