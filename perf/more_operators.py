"""Workloads of the microscaled 4-bit operators and of the norm around a block:
the FP4 linear layer, weights quantised to 4 bits and back, and the residual
norm (post norm, gate, residual scale, next norm) that hands bf16, e4m3 or
e2m1 operands to the next product.

`run` computes a case either in plain form (elementary torch operations in
fp32, rounded once at the end) or, with `own` set, by the library's calls;
`exact` computes it in 64 bits from the definitions. Sizes are those of the
block-FP8 models this library serves (dim 2048 / 5120 / 7168, inter 10944 /
18432, latent query rank 1536) and odd ones between.

e2m1 holds 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; element 2i of a row
is the low half of byte i. Formats: "e4m3" has a block scale in e4m3 for every
16 columns and an fp32 scale for every row; "ue8m0" a power of two for every 32
columns. The scale byte of (row, block) is at [row / 128, block / 4, row % 32,
row % 128 / 32, block % 4] of its tensor.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # One decoded token through the query up-projection: the weight is read once.
        {"name": "linear 1 of 24576x1536", "op": "linear", "M": 1, "N": 24576, "K": 1536, "fmt": "e4m3"},
        # A small decode batch: the benchmark's decode shape, rows that end inside a tile.
        {"name": "linear 8 of 10944x2048", "op": "linear", "M": 8, "N": 10944, "K": 2048, "fmt": "e4m3"},
        # An odd decode batch through an output projection, power-of-two scales.
        {"name": "linear 61 of 7168x2048 ue8m0", "op": "linear", "M": 61, "N": 7168, "K": 2048, "fmt": "ue8m0"},
        # A short prompt chunk of odd length.
        {"name": "linear 517 of 5120x7168", "op": "linear", "M": 517, "N": 5120, "K": 7168, "fmt": "e4m3"},
        # Prefill through the widest layer: the tensor cores.
        {"name": "linear 4096 of 18432x7168", "op": "linear", "M": 4096, "N": 18432, "K": 7168, "fmt": "e4m3"},
        # Prefill through its down-projection, power-of-two scales.
        {"name": "linear 4096 of 7168x18432 ue8m0", "op": "linear", "M": 4096, "N": 7168, "K": 18432, "fmt": "ue8m0"},
        # A checkpoint's weight to 4 bits, and back as the bf16 path uses it.
        {"name": "weight 18432x7168 fp32", "op": "weight", "M": 18432, "K": 7168, "fp32": True, "fmt": "e4m3"},
        # A narrow expert's weight of odd height, from bf16.
        {"name": "weight 1407x2048 ue8m0", "op": "weight", "M": 1407, "K": 2048, "fp32": False, "fmt": "ue8m0"},
        # One decoded token between two blocks: latency.
        {"name": "norm 1x7168", "op": "norm", "M": 1, "K": 7168, "out": "bf16", "post": False, "gate": "none",
         "scale": 1.0, "strided": False},
        # A prompt between two blocks with norms on both sides, into the FP8 product's operand: bandwidth.
        {"name": "norm 4099x7168 post to fp8", "op": "norm", "M": 4099, "K": 7168, "out": "fp8", "post": True,
         "gate": "column", "scale": 1.0, "strided": False},
        # A decode batch whose gate goes by the token, rows that are columns of a wider product.
        {"name": "norm 131x5120 gated", "op": "norm", "M": 131, "K": 5120, "out": "bf16", "post": True, "gate": "token",
         "scale": 0.5, "strided": True},
        # A decode step's seam: the norm writes the 4-bit operand, the latent down-projections read it.
        {"name": "step 16 of 2112x7168", "op": "step", "M": 16, "N": 2112, "K": 7168, "fmt": "e4m3", "post": False,
         "gate": "none", "scale": 1.0, "strided": False},
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is uniform over [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "weight", "norm", "norm", "step"])
    fmt = rng.choice(["e4m3", "ue8m0"])
    block = {"post": rng.random() < 0.5, "gate": rng.choice(["none", "column", "token"]),
             "scale": rng.choice([1.0, 1.0, 0.5, 1.4]), "strided": rng.random() < 0.3}
    while True:
        if op == "weight":
            c = {"op": op, "M": _log(rng, 16, 24576), "K": 128 * _log(rng, 1, 144), "fp32": rng.random() < 0.5, "fmt": fmt}
            if c["M"] * c["K"] <= 18432 * 7168:
                return c
            continue
        if op == "norm":
            out = rng.choice(["bf16", "bf16", "fp8"])
            unit = 128 if out == "fp8" else 8
            return {"op": op, "M": _log(rng, 1, 4099), "K": unit * _log(rng, max(1, 128 // unit), 7168 // unit),
                    "out": out, **block}
        if op == "step":
            return {"op": op, "M": _log(rng, 1, 256), "N": _log(rng, 64, 24576), "K": 128 * _log(rng, 4, 56), "fmt": fmt,
                    **block}
        c = {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, 24576), "K": 128 * _log(rng, 1, 144), "fmt": fmt}
        if c["M"] * c["N"] * c["K"] <= 4096 * 18432 * 7168 and c["N"] * c["K"] <= 18432 * 7168:
            return c


# ---- what a user's program has in hand ----------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 6949 + 29)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    st, M, K, op = dict(case), case["M"], case["K"], case["op"]
    if op == "weight":
        st["w"] = normal(M, K, std=0.02, dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        return st
    if op in ("linear", "step"):
        N, per = case["N"], 16 if case["fmt"] == "e4m3" else 32
        # codes of a normal weight whose block amax is 6: |w| / s is near a half normal of deviation 3.2
        v = normal(N, K, std=3.2)
        hi, lo = (_code_of(v[:, i::2]) for i in (1, 0))
        st["w"] = hi * 16 + lo
        rows, blocks = (N + 127) // 128 * 128, K // per
        if case["fmt"] == "e4m3":
            s = (300.0 + 140.0 * torch.rand((rows, blocks), generator=g, device=dev)).to(torch.float8_e4m3fn).view(torch.uint8)
            st["w_g"] = 0.02 / 3.2 / 370.0 * (0.9 + 0.2 * torch.rand(N, generator=g, device=dev))
        else:
            s = torch.randint(127 - 9, 127 - 6, (rows, blocks), generator=g, device=dev).to(torch.uint8)
            st["w_g"] = None
        s[N:] = 0
        st["values"] = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=dev)
        st["w_s"] = s.view(rows // 128, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    if op == "linear":
        st["x"] = normal(M, K)
        st["x"][:, torch.randperm(K, generator=g, device=dev)[:max(1, K // 100)]] *= 20      # outlier channels
        return st
    wide = 640 if case["strided"] else 0
    st["y"] = normal(M, K + wide)[:, wide:]
    st["x"] = normal(M, K, std=4.0)
    st["norm_w"] = 1.0 + normal(K, std=0.1, dtype=torch.float32)
    st["post_w"] = 0.7 + normal(K, std=0.1, dtype=torch.float32) if case["post"] else None
    st["gate_w"] = {"none": lambda: None, "column": lambda: 0.5 + normal(K, std=0.1, dtype=torch.float32),
                    "token": lambda: normal(M, K, std=0.5)}[case["gate"]]()
    return st


def _code_of(v):
    """The e2m1 codes of v (nearest, ties to the even code, saturating)."""
    a = v.float().abs()
    up = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    at = torch.bucketize(a, up) + ((a == 0.75) | (a == 1.75) | (a == 3.5)).int()
    return (at + 8 * (v < 0)).to(torch.uint8)


# ---- one pass -------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"linear": _plain_linear, "weight": _plain_weight, "norm": _plain_norm, "step": _plain_step}[st["op"]](st)


def _run_own(st):
    import fp8_block_scaled_quant_gb300 as fb

    op = st["op"]
    if op == "norm":
        r, h = fb.residual_norm(st["y"], st["x"], st["norm_w"], post_w=st["post_w"], gate=st["gate_w"],
                                residual_scale=st["scale"], eps=EPS, quant=None if st["out"] == "bf16" else "fp8")
        return {"r": r, "h": h} if st["out"] == "bf16" else {"r": r, "q": h[0], "s": h[1]}
    fmt = fb.FP4_E4M3 if st["fmt"] == "e4m3" else fb.FP4_UE8M0
    if op == "weight":
        return fb.fp4_dequant(*fb.fp4_quant(st["w"], fmt), fmt)
    if op == "linear":
        return fb.fp4_linear(st["x"], st["w"], st["w_s"], st["w_g"], fmt)
    r, h = fb.residual_norm(st["y"], st["x"], st["norm_w"], post_w=st["post_w"], gate=st["gate_w"],
                            residual_scale=st["scale"], eps=EPS, quant="fp4", scale_fmt=fmt)
    return {"r": r, "c": fb.fp4_gemm(*h, st["w"], st["w_s"], st["w_g"], fmt)}


def _plain_e2m1(v):
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _power_up(s):
    """The least power of two that is not below s, at least 2^-126."""
    m, e = torch.frexp(s)
    return torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e).clamp(min=-126))


def _plain_fp4(x, fmt):
    """The values that x stands for after quantisation to 4 bits."""
    if fmt == "ue8m0":
        b = x.unflatten(-1, (-1, 32))
        amax = b.abs().amax(-1, keepdim=True)
        s = _power_up(amax / torch.full_like(amax, 6.0))      # by a tensor: a true division
        return (_plain_e2m1(b / s) * s).flatten(-2)
    b = x.unflatten(-1, (-1, 16))
    amax = b.abs().amax(-1, keepdim=True)
    top = amax.amax(-2, keepdim=True).clamp(min=2.0 ** -100)
    g = top / torch.full_like(top, 2688.0)
    s = (amax * (torch.full_like(top, 448.0) / top)).to(torch.float8_e4m3fn).float()
    d = s * g
    r = torch.where(s > 0, torch.ones_like(d) / d, 0.0)
    return (_plain_e2m1(b * r) * s * g).flatten(-2)


def _plain_w(st):
    """The values of the 4-bit weight, fp32 [N, K]."""
    per = 16 if st["fmt"] == "e4m3" else 32
    v = st["values"][torch.stack([st["w"] & 15, st["w"] >> 4], -1).flatten(-2).int()]
    s = st["w_s"].permute(0, 3, 2, 1, 4).flatten(3, 4).flatten(0, 2)[:st["N"]]
    if st["fmt"] == "e4m3":
        s = s.view(torch.float8_e4m3fn).float() * st["w_g"][:, None]
    else:
        s = torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.int() - 127)
    return (v.unflatten(-1, (-1, per)) * s[..., None]).flatten(-2)


def _plain_linear(st):
    return (_plain_fp4(st["x"].float(), st["fmt"]) @ _plain_w(st).t()).to(torch.bfloat16)


def _plain_weight(st):
    return _plain_fp4(st["w"].float(), st["fmt"]).to(torch.bfloat16)


def _rms(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w


def _plain_block(st):
    """(the new residual, its norm), fp32."""
    z = st["y"].float()
    if st["post_w"] is not None:
        z = _rms(z, st["post_w"])
    if st["gate_w"] is not None:
        z = z * st["gate_w"].float()
    r = st["x"].float() * st["scale"] + z
    return r, _rms(r, st["norm_w"])


def _plain_norm(st):
    r, h = _plain_block(st)
    if st["out"] == "bf16":
        return {"r": r.to(torch.bfloat16), "h": h.to(torch.bfloat16)}
    b = h.unflatten(-1, (-1, 128))
    s = b.abs().amax(-1, keepdim=True).clamp(min=1e-4)
    s = s / torch.full_like(s, 448.0)
    return {"r": r.to(torch.bfloat16), "q": (b / s).to(torch.float8_e4m3fn).flatten(-2), "s": s[..., 0]}


def _plain_step(st):
    r, h = _plain_block(st)
    return {"r": r.to(torch.bfloat16), "c": (_plain_fp4(h, st["fmt"]) @ _plain_w(st).t()).to(torch.bfloat16)}


# ---- the work of one pass ---------------------------------------------------------

def _fp4_bytes(n, fmt):
    return n // 2 + n // (16 if fmt == "e4m3" else 32)


def work(case):
    c = case
    M, K, op = c["M"], c["K"], c["op"]
    if op == "weight":
        # read once, the 4-bit weight written, its bf16 form written
        return {"bytes": M * K * (4 if c["fp32"] else 2) + _fp4_bytes(M * K, c["fmt"]) + M * K * 2, "flops": 4 * M * K}
    if op == "linear":
        N = c["N"]
        return {"bytes": M * K * 2 + _fp4_bytes(N * K, c["fmt"]) + 4 * N + M * N * 2, "flops": 2 * M * N * K}
    around = M * K * (6 + (2 if c["gate"] == "token" else 0)) + K * (4 + (4 if c["post"] else 0) + (4 if c["gate"] == "column" else 0))
    if op == "norm":
        return {"bytes": around + (2 * M * K if c["out"] == "bf16" else M * K + M * K // 32), "flops": 10 * M * K}
    N = c["N"]
    return {"bytes": around + _fp4_bytes(N * K, c["fmt"]) + 4 * N + M * N * 2, "flops": 2 * M * N * K + 10 * M * K}


# ---- the definitions in 64 bits -----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "weight":
        v, s, g = _quant64(st["w"].double(), case["fmt"])
        out = v.view(case["M"], s.shape[1], -1) * s[..., None] * g[:, None, None]
        return out.view(case["M"], -1)
    if case["op"] == "linear":
        return _product64(_quant64(st["x"].double(), case["fmt"]), _weight64(st))
    y = st["y"].double()
    if case["post"]:
        y = y / (y.pow(2).sum(-1, keepdim=True) / case["K"] + EPS).sqrt() * st["post_w"].double()
    if case["gate"] != "none":
        y = y * st["gate_w"].double()
    r = y + st["x"].double() * case["scale"]
    h = r / (r.pow(2).sum(-1, keepdim=True) / case["K"] + EPS).sqrt() * st["norm_w"].double()
    if case["op"] == "step":
        return {"r": r, "c": _product64(_quant64(h, case["fmt"]), _weight64(st))}
    if case["out"] == "bf16":
        return {"r": r, "h": h}
    hb = h.view(case["M"], -1, 128)
    s = hb.abs().amax(-1).clamp(min=1e-4) / 448.0
    v = (hb / s[..., None]).abs()
    step = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    q = torch.copysign((torch.round(v / step) * step).clamp(max=448.0), hb)
    return {"r": r, "q": q.view(h.shape), "s": s}


VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest64(v):
    """The nearest e2m1 value of v; halfway, the one with the even code."""
    a = v.abs()
    out = torch.zeros_like(a)
    for i in range(1, 8):
        mid = (VALUES[i - 1] + VALUES[i]) / 2
        out[(a > mid) if i % 2 else (a >= mid)] = VALUES[i]
    return torch.copysign(out, v)


def _quant64(x, fmt):
    """(e2m1 values [M, K], block scales [M, blocks], row scales [M]), all in 64 bits. The rule rounds each of
    its scales to fp32 (or to the scale's type): values sit on borders between two codes, where that decides."""
    f32 = lambda t: t.float().double()  # noqa: E731
    if fmt == "ue8m0":
        b = x.view(x.shape[0], -1, 32)
        s = torch.exp2(torch.ceil(torch.log2(f32(b.abs().amax(-1) / 6.0))).clamp(min=-126))
        return _nearest64(f32(b / s[..., None])).view(x.shape), s, torch.ones_like(x[:, 0])
    b = f32(x).view(x.shape[0], -1, 16)
    amax = b.abs().amax(-1)
    top = amax.amax(-1).clamp(min=2.0 ** -100)
    g = f32(top / 2688.0)
    t = f32(amax * f32(448.0 / top)[:, None]).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    s = torch.round(t / step) * step
    d = f32(s * g[:, None])
    r = torch.where(s > 0, f32(1.0 / d), 0.0)
    return _nearest64(f32(b * r[..., None])).view(x.shape), s, g


def _weight64(st):
    N, K, per = st["N"], st["K"], 16 if st["fmt"] == "e4m3" else 32
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), dtype=torch.float64, device="cuda")
    v = torch.empty((N, K), dtype=torch.float64, device="cuda")
    v[:, 0::2], v[:, 1::2] = table[(st["w"] % 16).long()], table[(st["w"] // 16).long()]
    row, block = torch.arange(N, device="cuda")[:, None], torch.arange(K // per, device="cuda")[None, :]
    byte = st["w_s"][row // 128, block // 4, row % 32, row % 128 // 32, block % 4]
    if st["fmt"] == "e4m3":
        return v, byte.view(torch.float8_e4m3fn).double(), st["w_g"].double()
    return v, torch.exp2(byte.double() - 127.0), torch.ones(N, dtype=torch.float64, device="cuda")


def _product64(a, w):
    """Sum over blocks of the scales' product times the codes' product: the
    latter a sum of at most 32 multiples of 1/4 below 36, exact in 32 bits."""
    (va, sa, ga), (vw, sw, gw) = a, w
    per = va.shape[1] // sa.shape[1]
    va, vw = va.float(), vw.float()
    out = torch.zeros((va.shape[0], vw.shape[0]), dtype=torch.float64, device=va.device)
    for b in range(sa.shape[1]):
        part = (va[:, b * per:(b + 1) * per] @ vw[:, b * per:(b + 1) * per].t()).double()
        out += part.mul_(sa[:, b, None]).mul_(sw[None, :, b])
    return out.mul_(ga[:, None]).mul_(gw[None, :])
