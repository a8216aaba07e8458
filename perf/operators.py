"""Workloads of the decode-step operators: the latent cache append with its
norm and rotations, the attention of single query tokens over a paged latent
cache with a shared prefix, and the whole mixture-of-experts layer for a few
tokens.

`run` computes a case either in plain form (elementary torch operations in
fp32, rounded once at the end) or, with `own` set, by the library's calls;
`exact` computes it in 64 bits from the definitions. Sizes are those of the
block-FP8 MLA / MoE models this library serves (latent 512 + 64 rotary
columns, 16 or 128 heads, 64 / 160 / 256 experts) and odd ones between.
"""
import math

import numpy as np
import torch

own = False

C, R, DN = 512, 64, 128     # latent columns, rotary columns, no-position columns of a query head
EPS = 1e-6
W_STD = 107.0               # e4m3 codes of a normal weight whose block amax maps to 448 sit near N(0, 107^2)


def listed():
    return [
        # One sequence that has just begun, 16 heads: nothing but latency.
        {"name": "attn 1x16 own 9", "op": "attention", "B": 1, "H": 16, "P": 0, "own": 9, "ragged": False, "page": 64},
        # One long conversation, 128 heads: one row tile, work split over the key axis.
        {"name": "attn 1x128 own 32768", "op": "attention", "B": 1, "H": 128, "P": 0, "own": 32768, "ragged": False,
         "page": 64},
        # A decode batch of ragged lengths, nothing shared: every key read once for 128 heads.
        {"name": "attn 32x128 own 8191", "op": "attention", "B": 32, "H": 128, "P": 0, "own": 8191, "ragged": True,
         "page": 64},
        # Few heads, an odd batch behind a system prompt of odd length, small pages.
        {"name": "attn 61x16 prefix 2011 own 257", "op": "attention", "B": 61, "H": 16, "P": 2011, "own": 257,
         "ragged": True, "page": 16},
        # Many requests behind one long document: the prefix is a matrix product over all rows.
        {"name": "attn 64x128 prefix 32768 own 511", "op": "attention", "B": 64, "H": 128, "P": 32768, "own": 511,
         "ragged": True, "page": 64},
        # One decoded token appended, 128 heads: latency.
        {"name": "append 1x128", "op": "append", "T": 1, "H": 128, "page": 64, "strided": False},
        # A decode batch, 16 heads, rows that are columns of a wider product.
        {"name": "append 129x16 strided", "op": "append", "T": 129, "H": 16, "page": 16, "strided": True},
        # A prompt written at once: bandwidth.
        {"name": "append 6151x128", "op": "append", "T": 6151, "H": 128, "page": 64, "strided": False},
        # One token through 256 experts of the largest model: eight experts and the shared one are read.
        {"name": "moe 1 of 7168x2048 E256", "op": "moe", "T": 1, "dim": 7168, "inter": 2048, "E": 256, "k": 8, "ns": 1,
         "groups": 8, "kept": 4, "sigmoid": True, "bias": True, "ue8m0": False},
        # Five tokens of a small model (64 narrow experts, softmax gate, two shared).
        {"name": "moe 5 of 2048x1408 E64", "op": "moe", "T": 5, "dim": 2048, "inter": 1408, "E": 64, "k": 6, "ns": 2,
         "groups": 1, "kept": 1, "sigmoid": False, "bias": False, "ue8m0": False},
        # A decode batch of the largest model, power-of-two scales.
        {"name": "moe 16 of 7168x2048 E256 ue8m0", "op": "moe", "T": 16, "dim": 7168, "inter": 2048, "E": 256, "k": 8,
         "ns": 1, "groups": 8, "kept": 4, "sigmoid": True, "bias": True, "ue8m0": True},
        # The most tokens the layer takes, middle-sized experts.
        {"name": "moe 32 of 5120x1536 E160", "op": "moe", "T": 32, "dim": 5120, "inter": 1536, "E": 160, "k": 6,
         "ns": 2, "groups": 8, "kept": 3, "sigmoid": False, "bias": False, "ue8m0": False},
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is uniform over [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "moe", "moe"])
    if op == "append":
        return {"op": op, "T": _log(rng, 1, 6151), "H": rng.choice([1, 5, 16, 32, 40, 64, 128]),
                "page": rng.choice([16, 32, 64, 128]), "strided": rng.random() < 0.5}
    if op == "attention":
        while True:
            c = {"op": op, "B": _log(rng, 1, 128), "H": rng.choice([1, 7, 16, 24, 32, 64, 128]),
                 "P": rng.choice([0, _log(rng, 1, 32768)]), "own": _log(rng, 1, 32768), "ragged": rng.random() < 0.8,
                 "page": rng.choice([16, 32, 64, 128])}
            if c["B"] * c["H"] * (c["P"] + c["own"]) <= 1 << 28 and c["B"] * c["own"] <= 1 << 18 and 3072 not in c.values():
                return c
    while True:
        E = 32 * rng.randint(1, 8)
        c = {"op": op, "T": _log(rng, 1, 32), "dim": 256 * _log(rng, 4, 28), "inter": 128 * _log(rng, 2, 16), "E": E,
             "k": rng.randint(1, 8), "ns": rng.randint(0, 2), "groups": 1, "kept": 1, "sigmoid": rng.random() < 0.5,
             "bias": rng.random() < 0.5, "ue8m0": rng.random() < 0.3}
        if rng.random() < 0.5:
            c["groups"], c["kept"] = 4, rng.randint(2, 3)
        if (E + 2) * c["dim"] * c["inter"] <= 258 * 7168 * 2048 and 3072 not in c.values() and \
                c["T"] * (c["k"] + c["ns"]) * c["dim"] * c["inter"] <= 144 * 7168 * 2048:
            return c


# ---- what a user's program has in hand ----------------------------------------

def _lens(c):
    """Own lengths of a batch: all equal, or ragged down to zero (fixed by the
    case: the lengths are part of the workload)."""
    B, L = c["B"], c["own"]
    if not c["ragged"]:
        return [L] * B
    r = np.random.RandomState(1000 + 7 * B + L)
    v = [int(x) for x in r.randint(0, L + 1, size=B)]
    v[r.randint(0, B)] = L
    return v


def _rope_table(n, dev):
    """cos and sin of position * 10000^(-2i/64), fp32 [n, 32, 2]."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
    a = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    st = dict(case)
    if case["op"] == "append":
        T, H, ps = case["T"], case["H"], case["page"]
        pages = 2 * ((T + ps - 1) // ps) + 3
        wide = 640 if case["strided"] else 0
        kv = normal(T, C + R + wide)
        q = normal(T, H * (DN + R) + wide)
        st["kv"] = kv[:, wide:]
        st["q"] = q[:, wide:].view(T, H, DN + R)
        st["norm_w"] = 1.0 + normal(C, std=0.1, dtype=torch.float32)
        st["rope"] = _rope_table(8192, dev)
        st["positions"] = torch.randint(0, 8192, (T,), generator=g, device=dev)
        st["slots"] = torch.randperm(pages * ps, generator=g, device=dev)[:T].contiguous()
        if T > 2:
            st["slots"][T // 2] = -1          # a padding token of the batch
        st["cache"] = normal(pages, ps, C + R)
        return st
    if case["op"] == "attention":
        B, H, P, ps = case["B"], case["H"], case["P"], case["page"]
        lens = _lens(case)
        npp, npo = (P + ps - 1) // ps, max(1, (max(lens) + ps - 1) // ps)
        per = [(n + ps - 1) // ps for n in lens]
        total = npp + sum(per) + 2
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        table = torch.zeros((B, npo), dtype=torch.int32, device=dev)
        have = torch.arange(npo, device=dev)[None, :] < torch.tensor(per, device=dev)[:, None]
        table[have] = ids[npp: npp + sum(per)]
        st["cache"] = torch.empty((total, ps, C + R), dtype=torch.bfloat16, device=dev)
        for p0 in range(0, total, 4096):      # in parts: the fp32 draw of a long cache is large
            n = min(4096, total - p0)
            st["cache"][p0:p0 + n] = normal(n, ps, C + R)
        st["prefix_pages"] = ids[:npp].contiguous()
        st["table"] = table
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["q"], st["q_pe"] = normal(B, H, C), normal(B, H, R)
        st["scale"] = (DN + R) ** -0.5
        return st
    T, dim, inter, E, K = case["T"], case["dim"], case["inter"], case["E"], case["E"] + case["ns"]
    st["x"] = normal(T, dim)
    st["gate_w"] = normal(E, dim, std=dim ** -0.5)
    st["gate_bias"] = normal(E, std=0.1, dtype=torch.float32) if case["bias"] else None
    for name, n, k in (("w1", inter, dim), ("w3", inter, dim), ("w2", dim, inter)):
        w = torch.empty((K * n, k), dtype=torch.float8_e4m3fn, device=dev)
        for e in range(0, K, 8):
            m = min(8, K - e) * n
            v = torch.randn((m, k), generator=g, device=dev, dtype=torch.bfloat16)
            w[e * n:e * n + m] = v.mul_(W_STD).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s = 0.02 / W_STD * (0.8 + 0.4 * torch.rand((K * n // 128, k // 128), generator=g, device=dev))
        st[name], st[name + "_s"] = w, _power_of_two(s) if case["ue8m0"] else s
    return st


def _power_of_two(s):
    """The least power of two that is not below s."""
    m, e = torch.frexp(s)
    return torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))


# ---- one pass -------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"append": _plain_append, "attention": _plain_attention, "moe": _plain_moe}[st["op"]](st)


def _run_own(st):
    import fp8_block_scaled_quant_gb300 as fb

    if st["op"] == "append":
        qn, qp = fb.mla_append(st["kv"], st["norm_w"], st["rope"], st["positions"], st["slots"], st["cache"],
                               q=st["q"], eps=EPS)
        return {"cache": st["cache"], "q_nope": qn, "q_pe": qp}
    if st["op"] == "attention":
        return fb.mla_attention(st["q"], st["q_pe"], st["cache"], st["table"], st["lens"], st["scale"],
                                prefix_pages=st["prefix_pages"], prefix_len=st["P"])
    return fb.moe_layer(st["x"], st["gate_w"], st["w1"], st["w1_s"], st["w3"], st["w3_s"], st["w2"], st["w2_s"],
                        topk=st["k"], gate_bias=st["gate_bias"], n_groups=st["groups"], topk_groups=st["kept"],
                        score_func=fb.SCORE_SIGMOID if st["sigmoid"] else fb.SCORE_SOFTMAX, route_scale=2.5,
                        n_shared=st["ns"], scale_fmt=fb.SCALE_UE8M0 if st["ue8m0"] else fb.SCALE_FP32)


def _rotate(x, cs):
    """Pairs (x[2i], x[2i+1]) turned by the angle whose cos and sin are cs[..., i, :]."""
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cs[..., 0], cs[..., 1]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _plain_append(st):
    kv, q = st["kv"].float(), st["q"].float()
    lat = kv[:, :C]
    lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * st["norm_w"]
    cs = st["rope"][st["positions"]]
    row = torch.cat([lat, _rotate(kv[:, C:], cs)], -1).to(torch.bfloat16)
    cache, slots = st["cache"], st["slots"]
    flat = cache.view(-1, C + R)
    keep = slots >= 0
    at = slots.clamp(min=0)
    # A padding token writes nothing: every token writes its slot's row, and a
    # padding token's write repeats what the first kept token writes.
    first = keep.to(torch.int8).argmax()
    flat[torch.where(keep, at, at[first])] = torch.where(keep[:, None], row, row[first])
    return {"cache": cache, "q_nope": st["q"][..., :DN].contiguous(),
            "q_pe": _rotate(q[..., DN:], cs[:, None]).to(torch.bfloat16)}


def _plain_attention(st):
    P, ps, lens = st["P"], st["page"], st["lens"]
    q = torch.cat([st["q"], st["q_pe"]], -1).float()
    own_rows = st["cache"][st["table"].long()].flatten(1, 2)
    there = torch.arange(own_rows.shape[1], device=q.device)[None, :] < lens[:, None]
    kv_o = torch.where(there[..., None], own_rows, 0).float()
    kv_p = st["cache"][st["prefix_pages"].long()].view(-1, C + R)[:P].float()
    s_o = torch.einsum("bhc,blc->bhl", q, kv_o).mul_(st["scale"]).masked_fill_(~there[:, None], -math.inf)
    s = torch.cat([torch.einsum("bhc,kc->bhk", q, kv_p).mul_(st["scale"]), s_o], -1)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhk,kc->bhc", p[..., :P], kv_p[:, :C]) + torch.einsum("bhl,blc->bhc", p[..., P:], kv_o[..., :C])
    return torch.where(l > 0, o / l, 0.0).to(torch.bfloat16)


def _plain_quant(v, ue8m0):
    """Values of v [..., K] after quantisation to e4m3 by blocks of 128."""
    b = v.unflatten(-1, (-1, 128))
    s = b.abs().amax(-1, keepdim=True).clamp(min=1e-4)
    s = s / torch.full_like(s, 448.0)      # by a tensor: a true division, not a product with 1 / 448
    s = _power_of_two(s) if ue8m0 else s
    return ((b / s).to(torch.float8_e4m3fn).float() * s).flatten(-2)


def _plain_gate(st, x):
    E, G = st["E"], st["groups"]
    logits = x @ st["gate_w"].float().t()
    if st["sigmoid"]:
        s = 1.0 / (1.0 + torch.exp(-logits))
    else:
        s = torch.exp(logits - logits.amax(-1, keepdim=True))
        s = s / s.sum(-1, keepdim=True)
    z = s + st["gate_bias"] if st["bias"] else s
    if G > 1:
        zg = z.unflatten(-1, (G, E // G))
        score = zg.sort(dim=-1, descending=True)[0][..., :2].sum(-1) if st["bias"] else zg.amax(-1)
        kept = score.sort(dim=-1, descending=True, stable=True)[1][:, :st["kept"]]
        mask = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        z = zg.masked_fill(~mask[..., None], -math.inf).flatten(-2)
    idx = z.sort(dim=-1, descending=True, stable=True)[1][:, :st["k"]]
    w = s.gather(1, idx)
    return idx, w / w.sum(-1, keepdim=True) * 2.5


def _plain_moe(st):
    T, E, ns = st["T"], st["E"], st["ns"]
    x = st["x"].float()
    idx, w = _plain_gate(st, x)
    shared = torch.arange(E, E + ns, device=x.device).expand(T, ns)
    ids, wt = torch.cat([idx, shared], 1), torch.cat([w, torch.ones((T, ns), device=x.device)], 1)
    xq = _plain_quant(x, st["ue8m0"])

    def weight(name):
        """The dequantised weight of every (token, slot) pair, [T, slots, n, k]."""
        q, s = st[name].view(E + ns, -1, st[name].shape[1]), st[name + "_s"].view(E + ns, -1, st[name + "_s"].shape[1])
        v = q.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
        return v.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128)).mul_(s[ids][..., :, None, :, None]).flatten(-2).flatten(-3, -2)

    h1 = torch.matmul(weight("w1"), xq[:, None, :, None])[..., 0]
    h3 = torch.matmul(weight("w3"), xq[:, None, :, None])[..., 0]
    u = _plain_quant(h1 / (1.0 + torch.exp(-h1)) * h3, st["ue8m0"])
    o = torch.matmul(weight("w2"), u[..., None])[..., 0]
    return (o * wt[..., None]).sum(1).to(torch.bfloat16)


# ---- the work of one pass ---------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "append":
        T, H = c["T"], c["H"]
        # kv row, slot, position and its rotation read, the cache row written; the queries read and written
        return {"bytes": T * (2 * (C + R) * 2 + 16 + R * 4 + 2 * H * (DN + R) * 2) + C * 4,
                "flops": T * (4 * C + 3 * R * (H + 1))}
    if c["op"] == "attention":
        B, H, P = c["B"], c["H"], c["P"]
        lens = _lens(c)
        keys = P + sum(lens)
        return {"bytes": keys * (C + R) * 2 + B * H * (2 * C + R) * 2 + 4 * B,
                "flops": 2 * H * (B * P + sum(lens)) * (C + R + C)}
    T, dim, inter, E, k, ns = c["T"], c["dim"], c["inter"], c["E"], c["k"], c["ns"]
    # each expert that a token is expected to reach is read once (codes and block scales)
    active = E * (1.0 - (1.0 - k / E) ** T) + ns
    return {"bytes": int(active * 3 * dim * inter * (1 + 4 / 16384) + E * dim * 2 + 2 * T * dim * 2),
            "flops": 2 * T * (3 * (k + ns) * dim * inter + E * dim)}


# ---- the definitions in 64 bits -----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "moe": _exact_moe}[case["op"]](st)


def _turn64(x, cs):
    z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous()) * torch.view_as_complex(cs.double())
    return torch.view_as_real(z).flatten(-2)


def _exact_append(st):
    cs = st["rope"][st["positions"]]
    cache = st["cache"].double().view(-1, C + R)
    kv = st["kv"].double()
    for at in (st["slots"] >= 0).nonzero()[:, 0].split(1024):
        v = kv[at, :C]
        norm = (v * v).sum(-1, keepdim=True).div(C).add(EPS).sqrt()
        cache[st["slots"][at]] = torch.cat([v / norm * st["norm_w"].double(), _turn64(kv[at, C:], cs[at])], -1)
    return {"cache": cache.view(st["cache"].shape), "q_nope": st["q"][..., :DN].double(),
            "q_pe": _turn64(st["q"][..., DN:], cs[:, None])}


def _exact_attention(st):
    B, H, P, ps = st["B"], st["H"], st["P"], st["page"]
    q = torch.cat([st["q"], st["q_pe"]], -1).double()
    lens = st["lens"].tolist()
    rows = st["cache"].view(-1, C + R)
    out = torch.zeros((B, H, C), dtype=torch.float64, device=q.device)
    pages = st["prefix_pages"].long()
    shared = rows[(pages[:, None] * ps + torch.arange(ps, device=q.device)).flatten()[:P]].double()
    for b in range(B):
        n = lens[b]
        at = (st["table"][b].long()[:, None] * ps + torch.arange(ps, device=q.device)).flatten()[:n]
        mine = rows[at].double()
        for h in range(0, H, 32):
            x = q[b, h:h + 32]
            s = torch.cat([x @ shared.t(), x @ mine.t()], 1) * st["scale"]
            if s.shape[1]:
                a = torch.softmax(s, 1)
                out[b, h:h + 32] = a[:, :P] @ shared[:, :C] + a[:, P:] @ mine[:, :C]
    return out


def _e4m3_64(v):
    """v rounded to the nearest e4m3 value (half to even), in 64 bits."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _quant64(v, ue8m0):
    # The rule divides in fp32 (scale and quotient each rounded once): bf16
    # values often sit exactly between two codes, where that rounding decides.
    b = v.reshape(v.shape[0], -1, 128)
    s = (b.abs().amax(-1, keepdim=True).clamp(min=1e-4) / 448.0).float().double()
    if ue8m0:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    return (_e4m3_64((b / s).float().double()) * s).reshape(v.shape)


def _exact_moe(st):
    T, E, ns, k, G = st["T"], st["E"], st["ns"], st["k"], st["groups"]
    x = st["x"].double()
    logits = x @ st["gate_w"].double().t()
    s = torch.sigmoid(logits) if st["sigmoid"] else torch.softmax(logits, -1)
    z = s + st["gate_bias"].double() if st["bias"] else s.clone()
    if G > 1:
        zg = z.view(T, G, E // G)
        best = zg.topk(2 if st["bias"] else 1, -1)[0].sum(-1)
        bar = best.topk(st["kept"], -1)[0][:, -1:]
        zg[best < bar] = -math.inf
    idx = z.topk(k, -1)[1]
    w = s.gather(1, idx)
    w = 2.5 * w / w.sum(-1, keepdim=True)
    xq = _quant64(x, st["ue8m0"])
    y = torch.zeros_like(x)

    def dense(name, e):
        n, kk = st[name].shape[0] // (E + ns), st[name].shape[1]
        sc = st[name + "_s"][e * n // 128:(e + 1) * n // 128].double()
        return st[name][e * n:(e + 1) * n].double().view(n // 128, 128, kk // 128, 128) \
            .mul_(sc[:, None, :, None]).view(n, kk)

    for e in sorted(set(idx.flatten().tolist())) + list(range(E, E + ns)):
        t, j = (idx == e).nonzero(as_tuple=True) if e < E else (torch.arange(T, device=x.device), None)
        h = xq[t] @ dense("w1", e).t()
        u = _quant64(h * torch.sigmoid(h) * (xq[t] @ dense("w3", e).t()), st["ue8m0"])
        o = u @ dense("w2", e).t()
        y[t] += o if j is None else o * w[t, j][:, None]
    return y
