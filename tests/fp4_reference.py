"""Plain forms of the 4-bit rules for the tests, in numpy: quantisation step by
step in fp32 (each numpy float32 operation is rounded to nearest even, as the
rule wants it), products in 64 bits."""
import numpy as np

E4M3, UE8M0 = 0, 1
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
MID = (VALUES[1:] + VALUES[:-1]) / 2


def e4m3_values():
    """The values of the codes 0 .. 0x7E (positive e4m3)."""
    c = np.arange(0x7F)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3_VALUES = e4m3_values()


def nearest(v, values):
    """Index of the nearest of the ascending `values`; halfway, the even index; above the last, the last."""
    mid = (values[1:] + values[:-1]) / 2
    i = np.searchsorted(mid, v, side="left")           # mid[i-1] < v <= mid[i]
    tie = (i < len(mid)) & (v == mid[np.minimum(i, len(mid) - 1)]) & (i % 2 == 1)
    return i + tie


def e2m1(v):
    """Codes of v: nearest, ties to the even code, saturating."""
    return (nearest(np.abs(v).astype(np.float64), VALUES) + 8 * np.signbit(v)).astype(np.uint8)


def quant(x, fmt):
    """x float32 [M, K] -> (codes [M, K], scale bytes [M, blocks], row scales float32 [M] or None)."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    f = np.float32
    with np.errstate(all="ignore"):
        if fmt == UE8M0:
            b = x.reshape(M, -1, 32)
            amax = np.abs(b).max(-1)
            bad = ~np.isfinite(amax)
            s = amax / f(6)
            m, e = np.frexp(np.where(bad, f(1), s))
            e = np.where(m == 0.5, e - 1, e)
            e = np.where(s == 0, -126, np.maximum(e, -126))
            v = np.where(bad[..., None], f(0), b * np.ldexp(f(1), -e)[..., None])
            return e2m1(v).reshape(M, K), np.where(bad, 255, e + 127).astype(np.uint8), None
        b = x.reshape(M, -1, 16)
        amax = np.abs(b).max(-1)
        top = np.abs(x).max(-1)
        bad = ~np.isfinite(top)
        a = np.maximum(np.where(bad, f(1), top), f(2.0 ** -100))
        g = a / f(2688)
        t = np.where(bad[:, None], f(0), amax) * (f(448) / a)[:, None]
        code = nearest(t.astype(np.float64), E4M3_VALUES)
        d = E4M3_VALUES[code].astype(f) * g[:, None]
        r = np.where(code > 0, f(1) / np.where(code > 0, d, f(1)), f(0))
        v = np.where((bad[:, None] | (code == 0))[..., None], f(0), b * r[..., None])
        codes = e2m1(v).reshape(M, K)
        return codes, code.astype(np.uint8), np.where(bad, f(np.nan), g)


def tiles(s):
    """Scale bytes [rows, blocks] in tile order, zeros after the last row."""
    rows, blocks = s.shape
    p = np.zeros(((rows + 127) // 128 * 128, blocks), np.uint8)
    p[:rows] = s
    return p.reshape(-1, 4, 32, blocks // 4, 4).transpose(0, 3, 2, 1, 4).copy()


def untiled(t, rows):
    """Scale bytes [rows, blocks] of scale tiles."""
    return t.transpose(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, -1)[:rows]


def unpack(q):
    """Codes [M, K] of bytes [M, K / 2]."""
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def values(codes, s, g, fmt):
    """float64 values of codes [M, K] with scale bytes [M, blocks]."""
    M, K = codes.shape
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    if fmt == UE8M0:
        sv = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    else:
        sv = E4M3_VALUES[s] * g.astype(np.float64)[:, None]
    return (v.reshape(M, s.shape[1], -1) * sv[..., None]).reshape(M, K)
