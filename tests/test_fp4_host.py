"""The 4-bit and norm entry points refuse what they cannot do before any launch (no GPU needed), and the tests' own
plain forms agree with each other."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import fp8_block_scaled_quant_gb300 as fb


@pytest.fixture(scope="module", autouse=True)
def built():
    from fp8_block_scaled_quant_gb300 import _build
    _build.build()


OK, NULL, SHAPE, ALIGN, WORKSPACE, ARG = 0, 1, 2, 3, 4, 8
P = 4096   # an aligned address that nothing reads


def test_quant_checks():
    f = fb._function("fp8blk_fp4_quant", "peiiiepppp")
    assert f(P, 0, 128, 4, 100, 0, P, P, P, None) == SHAPE
    assert f(P, 0, 127, 4, 128, 0, P, P, P, None) == SHAPE
    assert f(P, 0, 128, -1, 128, 0, P, P, P, None) == SHAPE
    assert f(P, 0, 128, 1 << 31, 128, 0, P, P, P, None) == SHAPE
    assert f(P, 2, 128, 4, 128, 0, P, P, P, None) == ARG
    assert f(P, 0, 128, 4, 128, 2, P, P, P, None) == ARG
    assert f(None, 0, 128, 0, 128, 0, None, None, None, None) == OK
    assert f(None, 0, 0, 3, 0, 0, None, None, None, None) == OK
    assert f(P, 0, 128, 4, 128, 0, P, P, None, None) == NULL
    assert f(None, 0, 128, 4, 128, 1, P, P, None, None) == NULL
    assert f(P + 2, 0, 128, 4, 128, 0, P, P, P, None) == ALIGN
    assert f(P, 0, 132, 4, 128, 0, P, P, P, None) == ALIGN
    assert f(P, 1, 130, 4, 128, 0, P, P, P, None) == ALIGN
    assert f(P, 0, 128, 4, 128, 0, P + 8, P, P, None) == ALIGN


def test_dequant_checks():
    f = fb._function("fp8blk_fp4_dequant", "pppiiepp")
    assert f(P, P, P, 4, 64, 0, P, None) == SHAPE
    assert f(P, P, P, 4, 128, 3, P, None) == ARG
    assert f(P, P, None, 4, 128, 0, P, None) == NULL
    assert f(P, P, P, 4, 128, 0, P + 2, None) == ALIGN
    assert f(None, None, None, 0, 128, 0, None, None) == OK


def test_gemm_checks():
    f = fb._function("fp8blk_fp4_gemm", "pppppppiiiep")
    assert f(P, P, P, P, P, P, P, 4, 4, 96, 0, None) == SHAPE
    assert f(P, P, P, P, P, P, P, 4, -4, 128, 0, None) == SHAPE
    assert f(P, P, P, P, P, P, P, 4, 1 << 29, 128, 0, None) == SHAPE
    assert f(P, P, P, P, P, P, P, 4, 4, 128, 5, None) == ARG
    assert f(P, P, None, P, P, P, P, 4, 4, 128, 0, None) == NULL
    assert f(P, P, P, P, P, None, P, 4, 4, 128, 0, None) == NULL
    assert f(P, P, P, P, P, P, None, 4, 4, 128, 0, None) == NULL
    assert f(P, P + 4, P, P, P, P, P, 4, 4, 128, 0, None) == ALIGN
    assert f(P, P, P, P + 8, P, P, P, 4, 4, 128, 0, None) == ALIGN
    assert f(P, P, P, P, P, P, P + 1, 4, 4, 128, 0, None) == ALIGN
    assert f(None, None, None, None, None, None, None, 0, 4, 128, 0, None) == OK
    assert f(None, None, None, None, None, None, None, 4, 4, 0, 0, None) == NULL


def test_linear_checks():
    f = fb._function("fp8blk_fp4_linear", "pippppiiiepzp")
    need = fb.fp4_linear_workspace_bytes(4, 64, 128)
    assert need >= 4 * 64 + 1024 + 16
    assert f(P, 128, P, P, P, P, 4, 64, 100, 0, P, need, None) == SHAPE
    assert f(P, 64, P, P, P, P, 4, 64, 128, 0, P, need, None) == SHAPE
    assert f(P, 128, P, P, P, P, 4, 64, 128, 2, P, need, None) == ARG
    assert f(P, 129, P, P, P, P, 4, 64, 128, 0, P, need, None) == ALIGN
    assert f(None, 128, P, P, P, P, 4, 64, 128, 0, P, need, None) == NULL
    assert f(P, 128, P, P, P, P, 4, 64, 128, 0, None, need, None) == WORKSPACE
    assert f(P, 128, P, P, P, P, 4, 64, 128, 0, P, need - 1, None) == WORKSPACE
    assert f(P, 128, P, P, P, P, 4, 64, 128, 0, P + 16, need, None) == ALIGN
    assert f(P, 128, P, P, P, P, 0, 64, 128, 0, None, 0, None) == OK


def test_norm_checks():
    f = fb._function("fp8blk_residual_norm", "pipipppifpfiieeppppp")

    def call(y=P, ys=128, x=P, xs=128, post=P, col=None, tok=None, gs=128, w=P, eps=1e-6, T=4, D=128, kind=0, fmt=0, r=P,
             h=P, hs=P, hg=P):
        return f(y, ys, x, xs, post, col, tok, gs, 1.0, w, eps, T, D, kind, fmt, r, h, hs, hg, None)

    assert call(kind=3) == ARG and call(kind=2, fmt=2) == ARG and call(kind=1, fmt=7) == ARG
    assert call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG and call(col=P, tok=P) == ARG
    assert call(D=100, ys=104, xs=104) == SHAPE and call(D=120, kind=1) == SHAPE and call(D=0) == SHAPE
    assert call(D=16392, ys=20000, xs=20000) == SHAPE and call(ys=120) == SHAPE and call(xs=64) == SHAPE
    assert call(tok=P, gs=8) == SHAPE and call(T=-1) == SHAPE
    assert call(y=None) == NULL and call(w=None) == NULL and call(h=None) == NULL
    assert call(kind=1, hs=None) == NULL and call(kind=2, hg=None) == NULL
    assert call(ys=129) == ALIGN and call(y=P + 2) == ALIGN and call(post=P + 4) == ALIGN and call(h=P + 8) == ALIGN
    assert call(kind=2, hs=P + 4) == ALIGN
    assert call(T=0, y=None, w=None, h=None) == OK


def test_scale_bytes():
    f = fb._function("fp8blk_fp4_scale_bytes", "iie", __import__("ctypes").c_size_t)
    for rows, K, fmt in ((1, 128, 0), (129, 384, 1), (0, 128, 0), (256, 7168, 0)):
        assert f(rows, K, fmt) == int(np.prod(fb.fp4_scale_shape(rows, K, fmt)))
    assert f(4, 100, 0) == 0


@pytest.mark.parametrize("call", [
    lambda t: fb.fp4_quant(t), lambda t: fb.fp4_linear(t, t.byte(), t.byte(), None),
    lambda t: fb.fp4_gemm(t.byte(), t.byte(), None, t.byte(), t.byte(), None),
    lambda t: fb.fp4_dequant(t.byte(), t.byte(), None), lambda t: fb.residual_norm(t, t, t[0].float())])
def test_host_tensors_are_refused(call):
    with pytest.raises(fb.Fp8BlkError):
        call(torch.zeros(4, 128, dtype=torch.bfloat16))


def test_reference_pins():
    """The plain form rounds e2m1 as its table says, e4m3 as torch does, and its tiles go there and back."""
    v = np.concatenate([ref.VALUES, ref.MID, np.nextafter(ref.MID, 0), np.nextafter(ref.MID, 9), [7.0, 1e9]])
    want = [0, 1, 2, 3, 4, 5, 6, 7] + [0, 2, 2, 4, 4, 6, 6] + [0, 1, 2, 3, 4, 5, 6] + [1, 2, 3, 4, 5, 6, 7] + [7, 7]
    assert ref.e2m1(v).tolist() == want
    assert ref.e2m1(-v).tolist() == [c + 8 for c in want]
    t = np.random.RandomState(0).uniform(0, 448, 20000).astype(np.float32) * np.exp2(-(np.arange(20000) % 20)).astype(np.float32)
    assert np.array_equal(ref.nearest(t.astype(np.float64), ref.E4M3_VALUES),
                          torch.from_numpy(t).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    s = np.random.RandomState(1).randint(0, 256, (300, 12)).astype(np.uint8)
    assert np.array_equal(ref.untiled(ref.tiles(s), 300), s)
    for row, block in ((0, 0), (131, 7), (299, 11)):
        assert ref.tiles(s)[row // 128, block // 4, row % 32, row % 128 // 32, block % 4] == s[row, block]
    c = np.random.RandomState(2).randint(0, 16, (3, 128)).astype(np.uint8)
    assert np.array_equal(ref.unpack(ref.pack(c)), c)
    # a quantised row is never further off than half a step of its largest block value
    x = np.random.RandomState(3).randn(5, 256).astype(np.float32)
    for fmt, per in ((ref.E4M3, 16), (ref.UE8M0, 32)):
        codes, sb, g = ref.quant(x, fmt)
        off = np.abs(ref.values(codes, sb, g, fmt) - x).reshape(5, -1, per).max(-1)
        assert np.all(off <= np.abs(x).reshape(5, -1, per).max(-1) * (0.22 if fmt == ref.E4M3 else 0.34))
