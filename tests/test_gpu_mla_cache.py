"""The latent cache append and the shared-prefix attention over the paged
latent cache, against the formulas in 64 bits.

Tolerances. u = 2^-8 is bf16's unit roundoff, r = 1.66e-3 its rms relative
rounding error (u / sqrt(3), averaged over a significand in [1, 2)).
Append: one rounding, u |ref|, after a few fp32 operations whose errors are
2^-20 of the magnitudes that go in.
Attention, per element: the output's rounding, u |out|; the weights' rounding,
u sum_j a_j |v_j - out| <= u (A + |out|) with A = sum_j a_j |v_j|; and the
scores' error d (fp32 sums of 576 products, at most 2^-16 of scale *
sum |x_i c_i|), 2 d A. Over a whole tensor of zero-mean values both roundings
are independent, so the error's norm is near sqrt(2) r = 2.3e-3 of the
output's norm; 4e-3 is allowed (one key too many or too few among 1000 moves
it by 3e-2)."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu
C, R, DN = 512, 64, 128
U = 2.0 ** -8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def rope_table(n):
    f = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


# ---- append -----------------------------------------------------------------------

def turn(x, cs):
    """(turned pairs, sum of the two products' magnitudes) in 64 bits."""
    a, b = x.double()[..., 0::2], x.double()[..., 1::2]
    c, s = cs[..., 0].double(), cs[..., 1].double()
    val = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    mag = torch.stack([(a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()], -1).flatten(-2)
    return val, mag


def check_append(T, H, page, strided, seed, with_q=True, pad=()):
    g = gen(seed)
    off = 64 if strided else 0
    kv = normal(g, T, C + R + 2 * off, std=3.0)[:, off:off + C + R]
    q = normal(g, T, H * (DN + R) + 2 * off)[:, off:off + H * (DN + R)].unflatten(1, (H, DN + R)) if with_q else None
    w = 1.0 + normal(g, C, std=0.2, dtype=torch.float32)
    rope = rope_table(777)
    pos = torch.randint(0, 777, (T,), generator=g, device="cuda")
    pages = (T + page - 1) // page + 2
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    for t in pad:
        slots[t] = -1 - t
    cache = normal(g, pages, page, C + R)
    before = cache.clone()
    kv0, q0 = kv.clone(), None if q is None else q.clone()
    got = fb.mla_append(kv, w, rope, pos, slots, cache, q=q, eps=1e-6)
    torch.cuda.synchronize()
    assert fb.last_device_error() == 0
    assert torch.equal(kv, kv0) and (q is None or torch.equal(q, q0))
    rows = cache.view(-1, C + R)
    kept = [t for t in range(T) if t not in pad]
    written = slots[kept]
    v = kv.double()[kept]
    lat = v[:, :C] / (v[:, :C].square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    cs = rope[pos]
    key, mag = turn(kv[kept][:, C:], cs[kept])
    assert ((rows[written][:, :C].double() - lat).abs() <= (U + 2.0 ** -18) * lat.abs()).all()
    assert ((rows[written][:, C:].double() - key).abs() <= U * key.abs() + 2.0 ** -20 * mag).all()
    rest = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
    rest[written] = False
    assert torch.equal(rows[rest].view(torch.int16), before.view(-1, C + R)[rest].view(torch.int16))
    if not with_q:
        assert got is None
        return
    qn, qp = got
    assert torch.equal(qn.view(torch.int16), q[..., :DN].contiguous().view(torch.int16))
    val, mag = turn(q[..., DN:], cs[:, None])
    assert ((qp.double() - val).abs() <= U * val.abs() + 2.0 ** -20 * mag).all()


@pytest.mark.parametrize("T,H,page,strided,pad", [
    (1, 128, 64, False, ()), (1, 1, 16, True, ()), (3, 7, 48, True, (1,)), (130, 16, 16, False, (0, 129)),
    (33, 40, 128, True, ()), (700, 128, 64, False, (5,)), (2000, 9, 32, True, ())])
def test_append(T, H, page, strided, pad):
    check_append(T, H, page, strided, 10 + T + H, pad=pad)


def test_append_without_queries():
    check_append(50, 1, 64, True, 3, with_q=False)


def test_append_takes_zero_rows_and_empty_batches():
    """A row of zeros normalises to zeros (eps), no token launches nothing."""
    cache = torch.full((1, 16, C + R), 7.0, dtype=torch.bfloat16, device="cuda")
    w, rope = torch.ones(C, device="cuda"), rope_table(4)
    kv = torch.zeros(1, C + R, dtype=torch.bfloat16, device="cuda")
    i64 = dict(dtype=torch.int64, device="cuda")
    fb.mla_append(kv, w, rope, torch.tensor([1], **i64), torch.tensor([3], **i64), cache)
    assert (cache[0, 3] == 0).all() and (cache[0, 2] == 7).all()
    fb.mla_append(kv[:0], w, rope, torch.zeros(0, **i64), torch.zeros(0, **i64), cache)
    assert fb.last_device_error() == 0


def test_append_reports_slots_and_positions_out_of_range():
    """They are checked on the device: nothing out of range is written, the
    error word says so, and the other tokens are appended."""
    cache = torch.zeros((2, 16, C + R), dtype=torch.bfloat16, device="cuda")
    w, rope = torch.ones(C, device="cuda"), rope_table(4)
    kv = normal(gen(1), 3, C + R)
    i64 = dict(dtype=torch.int64, device="cuda")
    fb.mla_append(kv, w, rope, torch.tensor([0, 1, 2], **i64), torch.tensor([32, 4, 1 << 40], **i64), cache)
    assert fb.last_device_error() == 0x100
    assert (cache.view(-1, C + R)[4] != 0).any() and (cache.view(-1, C + R)[5:] == 0).all()
    fb.mla_append(kv, w, rope, torch.tensor([0, -1, 4], **i64), torch.tensor([0, 1, 2], **i64), cache)
    assert fb.last_device_error() == 0x100


def test_append_slots_past_32_bit_offsets():
    """Row offsets beyond 2^31 elements (a 5 GB cache)."""
    page = 64
    pages = (1 << 31) // (page * (C + R)) + 40
    cache = torch.zeros((pages, page, C + R), dtype=torch.bfloat16, device="cuda")
    kv = normal(gen(2), 2, C + R)
    i64 = dict(dtype=torch.int64, device="cuda")
    last = pages * page - 1
    fb.mla_append(kv, torch.ones(C, device="cuda"), rope_table(4), torch.tensor([0, 0], **i64),
                  torch.tensor([last, 5], **i64), cache)
    rows = cache.view(-1, C + R)
    assert torch.equal(rows[last][C:].view(torch.int16), kv[0][C:].view(torch.int16))   # position 0: no turn
    assert torch.equal(rows[5][C:].view(torch.int16), kv[1][C:].view(torch.int16))
    assert (rows[last - 1] == 0).all() and fb.last_device_error() == 0


def test_append_refusals():
    cache = torch.zeros((2, 16, C + R), dtype=torch.bfloat16, device="cuda")
    w, rope = torch.ones(C, device="cuda"), rope_table(4)
    z = torch.zeros(2, dtype=torch.int64, device="cuda")
    kv = torch.zeros(2, C + R, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(2, C + R + 3, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(kv=kv.float()), dict(kv=kv[:, :500]), dict(w=w[:500]), dict(slots=z.int()), dict(slots=z[:1]),
                dict(kv=wide[:, :C + R]),                       # row stride not a multiple of 8 elements
                dict(cache=cache[:, :, :500]), dict(q=torch.zeros(2, 3, 100, dtype=torch.bfloat16, device="cuda")),
                dict(eps=-1.0), dict(eps=math.nan), dict(rope=rope[:, :16])):
        a = dict(kv=kv, w=w, rope=rope, pos=z, slots=z, cache=cache, q=None, eps=1e-6) | bad
        with pytest.raises(fb.Fp8BlkError):
            fb.mla_append(a["kv"], a["w"], a["rope"], a["pos"], a["slots"], a["cache"], q=a["q"], eps=a["eps"])


# ---- attention --------------------------------------------------------------------

def make_attention(B, H, P, lens, page, seed, std=1.0, spare=3):
    """Inputs whose every cache row outside the named lengths is NaN and whose
    unused table entries are nonsense."""
    g = gen(seed)
    npp = (P + page - 1) // page
    per = [(n + page - 1) // page for n in lens]
    total = npp + sum(per) + spare
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    prefix = ids[:npp].contiguous()
    table = torch.full((B, max(per + [1])), 1 << 30, dtype=torch.int32, device="cuda")
    cache = torch.full((total, page, C + R), math.nan, dtype=torch.bfloat16, device="cuda")
    rows = cache.view(-1, C + R)

    def at(pages, n):
        k = torch.arange(n, device="cuda")
        return pages.long()[k // page] * page + k % page

    keys_p = at(prefix, P) if P else torch.zeros(0, dtype=torch.int64, device="cuda")
    rows[keys_p] = normal(g, P, C + R)
    keys_o, k = [], npp
    for b in range(B):
        table[b, :per[b]] = ids[k:k + per[b]]
        keys_o.append(at(table[b], lens[b]) if lens[b] else keys_p[:0])
        rows[keys_o[b]] = normal(g, lens[b], C + R)
        k += per[b]
    return dict(q=normal(g, B, H, C, std=std), q_pe=normal(g, B, H, R, std=std), cache=cache, prefix=prefix, P=P,
                table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), keys_p=keys_p, keys_o=keys_o,
                scale=(DN + R) ** -0.5)


def call_attention(a, lse=None, **kw):
    return fb.mla_attention(a["q"], a["q_pe"], a["cache"], a["table"], a["lens"], a["scale"],
                            prefix_pages=a["prefix"], prefix_len=a["P"], lse=lse, **kw)


def check_attention(a, out, lse, requests=None, norm=True):
    B, H = a["q"].shape[:2]
    rows = a["cache"].view(-1, C + R)
    err2 = ref2 = 0.0
    for b in range(B) if requests is None else requests:
        keys = torch.cat([a["keys_p"], a["keys_o"][b]])
        if not len(keys):
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        x = torch.cat([a["q"][b], a["q_pe"][b]], -1).double()
        kv = rows[keys].double()
        s = x @ kv.t() * a["scale"]
        d = 2.0 ** -16 * a["scale"] * (x.abs() @ kv.abs().t()).amax(-1, keepdim=True)
        w = torch.softmax(s, -1)
        ref = w @ kv[:, :C]
        A = w @ kv[:, :C].abs()
        e = (out[b].double() - ref).abs()
        assert (e <= (2 * U) * ref.abs() + (U + 2 * d) * A).all(), f"request {b}: {e.max()}"
        l64 = torch.logsumexp(s, -1)
        assert ((lse[b].double() - l64).abs() <= d[:, 0] + U / 4 + 1e-6 * l64.abs()).all()
        err2 += float(e.square().sum())
        ref2 += float(ref.square().sum())
    if norm and ref2:
        assert math.sqrt(err2 / ref2) <= 4e-3, math.sqrt(err2 / ref2)


CASES = [
    # B, H, prefix, lens, page
    (1, 16, 0, [9], 64),
    (1, 128, 0, [1], 64),
    (1, 1, 0, [0], 16),
    (2, 128, 0, [0, 130], 64),
    (3, 128, 100, [0, 1, 300], 32),
    (1, 128, 129, [0], 16),
    (5, 16, 0, [1, 15, 16, 17, 0], 16),
    (5, 16, 1, [63, 64, 65, 0, 129], 64),
    (9, 7, 200, [5, 0, 128, 127, 1, 33, 31, 32, 300], 16),
    (4, 20, 128, [7, 255, 256, 257], 48),
    (3, 64, 1000, [40, 0, 1000], 128),
    (2, 130, 77, [90, 500], 64),
    (2, 256, 300, [10, 200], 32),
    (1, 128, 0, [5000], 64),
    (1, 5, 0, [9000], 16),
    (2, 40, 6000, [100, 3], 64),
    (300, 16, 300, [(37 * i) % 90 for i in range(300)], 16),
    (40, 128, 500, [(371 * i) % 700 for i in range(40)], 64),
]


@pytest.mark.parametrize("B,H,P,lens,page", CASES, ids=[f"B{c[0]}-H{c[1]}-P{c[2]}-{max(c[3])}-page{c[4]}" for c in CASES])
def test_attention(B, H, P, lens, page):
    a = make_attention(B, H, P, lens, page, 100 + B + H + P)
    lse = torch.full((B, H), 5.0, device="cuda")
    out = call_attention(a, lse)
    torch.cuda.synchronize()
    assert fb.last_device_error() == 0
    check_attention(a, out, lse)
    again = call_attention(a)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))   # a fixed order of every sum


@pytest.mark.parametrize("std", [0.01, 30.0])
def test_attention_flat_and_peaked_weights(std):
    """Nearly equal weights, and weights that a few keys dominate (running
    maxima that keep rising)."""
    a = make_attention(3, 128, 700, [800, 0, 33], 64, 7, std=std)
    lse = torch.empty((3, 128), device="cuda")
    out = call_attention(a, lse)
    check_attention(a, out, lse, norm=std < 1)
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("H", [16, 128])
def test_attention_rising_scores(H):
    """Keys sorted so that every tile's maximum passes the last one by far
    more than the step at which the output is rescaled, then falling ones."""
    a = make_attention(2, H, 640, [640, 300], 64, 8)
    rows = a["cache"].view(-1, C + R)
    a["q"].zero_()
    a["q"][:, :, 0] = 8.0
    up = torch.arange(640, device="cuda") // 4 * 1.0
    rows[a["keys_p"], 0] = up.to(torch.bfloat16)
    rows[a["keys_o"][0], 0] = (up + 160).to(torch.bfloat16)
    rows[a["keys_o"][1], 0] = (100 - up[:300]).to(torch.bfloat16)
    lse = torch.empty((2, H), device="cuda")
    out = call_attention(a, lse)
    check_attention(a, out, lse, norm=False)


def test_attention_of_equal_keys_is_the_key():
    """All keys alike: the weights' roundings cancel and the output is the
    latent itself, whatever the length."""
    a = make_attention(2, 16, 300, [0, 1000], 16, 9)
    row = normal(gen(4), C + R)
    a["cache"].view(-1, C + R)[:] = row
    out = call_attention(a)
    assert ((out.double() - row[:C].double()).abs() <= 2.0 ** -20 * row[:C].double().abs()).all()


def test_attention_bad_values_stay_with_their_request():
    """Inf and NaN among one request's own keys make that request's rows NaN,
    not those of requests that share its row tile."""
    a = make_attention(4, 16, 200, [40, 50, 60, 70], 16, 10)
    clean = call_attention(a)
    rows = a["cache"].view(-1, C + R)
    rows[a["keys_o"][1][7]] = math.nan
    rows[a["keys_o"][2][9], 3] = math.inf
    out = call_attention(a)
    assert out[1].isnan().all() and out[2][:, 3].float().abs().amax() > 1e30 or out[2][:, 3].isnan().any()
    for b in (0, 3):
        assert torch.equal(out[b].view(torch.int16), clean[b].view(torch.int16))


def test_attention_splitting_the_keys_leaves_the_result():
    """The same keys as prefix, as own keys, or as some of each."""
    base = make_attention(1, 128, 0, [4096], 64, 11)
    ref = call_attention(base).double()
    for cut in (64, 2048, 4032):
        a = dict(base)
        a["P"], a["prefix"] = cut, base["table"][0, :cut // 64].contiguous()
        a["table"] = base["table"][:, cut // 64:].contiguous()
        a["lens"] = base["lens"] - cut
        got = call_attention(a).double()
        assert float((got - ref).norm() / ref.norm()) <= 4e-3


def test_attention_ids_and_lengths_out_of_range():
    """A page id outside the cache reads as zeros and is reported; lengths are
    taken as the nearer end of their range."""
    a = make_attention(2, 16, 0, [64, 64], 16, 12)
    a["table"][1, 2] = a["cache"].shape[0]
    call_attention(a)
    assert fb.last_device_error() == 0x100
    a["table"][1, 2] = -5
    call_attention(a)
    assert fb.last_device_error() == 0x100
    a = make_attention(2, 16, 0, [64, 64], 16, 12)
    ref = call_attention(a)
    a["lens"].copy_(torch.tensor([1000, 64]))
    assert torch.equal(call_attention(a).view(torch.int16), ref.view(torch.int16))
    a["lens"].copy_(torch.tensor([-3, 64]))
    assert (call_attention(a)[0] == 0).all()
    assert fb.last_device_error() == 0


def test_attention_empty_batch_and_empty_cache():
    a = make_attention(2, 16, 0, [0, 0], 16, 13)
    e = dict(dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, 16), device="cuda")
    out = fb.mla_attention(a["q"], a["q_pe"], torch.empty((0, 16, C + R), **e),
                           torch.zeros((2, 0), dtype=torch.int32, device="cuda"), a["lens"], 0.1, lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all()
    out = fb.mla_attention(a["q"][:0], a["q_pe"][:0], a["cache"], a["table"][:0], a["lens"][:0], 0.1)
    assert out.shape == (0, 16, C) and fb.last_device_error() == 0


def test_attention_pages_past_32_bit_offsets():
    page = 64
    pages = (1 << 31) // (page * (C + R)) + 40
    cache = torch.empty((pages, page, C + R), dtype=torch.bfloat16, device="cuda")
    small = make_attention(1, 16, 0, [100], page, 14)
    ids = torch.tensor([[pages - 1, pages - 30]], dtype=torch.int32, device="cuda")
    for k in range(2):
        cache[ids[0, k].item()] = small["cache"][small["table"][0, k].item()]
    got = fb.mla_attention(small["q"], small["q_pe"], cache, ids, small["lens"], small["scale"])
    assert torch.equal(got.view(torch.int16), call_attention(small).view(torch.int16))
    assert fb.last_device_error() == 0


def test_attention_workspace_and_streams():
    """A workspace of garbage gives the same bits; calls on a side stream are
    ordered there."""
    a = make_attention(5, 16, 300, [200, 0, 5, 700, 64], 16, 15)
    ref = call_attention(a)
    n = fb.mla_attention_workspace_bytes(5, 16, 300)
    buf = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[(-buf.data_ptr()) % 256:][:n]
    assert torch.equal(call_attention(a, ws=ws).view(torch.int16), ref.view(torch.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [call_attention(a) for _ in range(3)]
    side.synchronize()
    for o in got:
        assert torch.equal(o.view(torch.int16), ref.view(torch.int16))
    with pytest.raises(fb.Fp8BlkError):
        call_attention(a, ws=ws[:n - 1])


def test_attention_in_a_graph_reads_new_lengths():
    a = make_attention(2, 128, 100, [300, 200], 64, 16)
    out = torch.empty((2, 128, C), dtype=torch.bfloat16, device="cuda")
    full = call_attention(a)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call_attention(a, out=out)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call_attention(a, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), full.view(torch.int16))
    a["lens"].copy_(torch.tensor([7, 0]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), call_attention(a).view(torch.int16))


def test_append_then_attention():
    """A decode step: the appended rows are read by the next call on the stream."""
    g = gen(17)
    B, H, page = 4, 16, 16
    a = make_attention(B, H, 64, [17, 33, 1, 48], page, 18)
    kv, q = normal(g, B, C + R), normal(g, B, H, DN + R)
    w, rope = torch.ones(C, device="cuda"), rope_table(200)
    pos = a["lens"].long() + 63
    slots = torch.stack([k[-1] for k in a["keys_o"]])
    step = dict(a, cache=a["cache"].clone())
    _, q_pe = fb.mla_append(kv, w, rope, pos, slots, step["cache"], q=q)
    got = fb.mla_attention(a["q"], q_pe, step["cache"], a["table"], a["lens"], a["scale"], prefix_pages=a["prefix"],
                           prefix_len=64)
    torch.cuda.synchronize()
    lse = torch.empty((B, H), device="cuda")
    step["q_pe"] = q_pe
    again = call_attention(step, lse)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    check_attention(step, again, lse)
    assert not torch.equal(call_attention(dict(a, q_pe=q_pe)).view(torch.int16), got.view(torch.int16))


def test_attention_refusals():
    a = make_attention(2, 16, 32, [20, 30], 16, 19)
    i32 = torch.int32
    for bad in (dict(q=a["q"].float()), dict(q=a["q"][:, :, :500]), dict(q_pe=a["q_pe"][:1]),
                dict(cache=a["cache"][:, :8].contiguous()),          # page size not a multiple of 16
                dict(table=a["table"].long()), dict(lens=a["lens"][:1]), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(P=33), dict(prefix=None),
                dict(q=a["q"].cpu()), dict(q=a["q"].transpose(0, 1))):
        with pytest.raises(fb.Fp8BlkError):
            call_attention(a | bad)
    with pytest.raises(fb.Fp8BlkError):
        call_attention(a, out=torch.empty((2, 16, 500), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fb.Fp8BlkError):
        call_attention(a, lse=torch.empty((2, 15), device="cuda"))
    assert fb.mla_attention_workspace_bytes(-1, 16, 0) == 0 and fb.mla_attention_workspace_bytes(1, 0, 0) == 0
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("H", [7, 16, 128, 130])
@pytest.mark.parametrize("stride", [1, 9])
def test_attention_without_any_key(H, stride):
    """No prefix and every length zero: zeros and -inf, whether or not rows can have several parts (stride pages of
    64 keys). The lengths are on the device, so the host launches as for any batch. Shared memory was used by a call
    with keys before."""
    a = make_attention(5, H, 0, [64 * stride] * 5, 64, 23)
    for _ in range(3):
        call_attention(a)
        lse = torch.full((5, H), 5.0, device="cuda")
        out = call_attention(dict(a, lens=torch.zeros_like(a["lens"])), lse)
        assert (out == 0).all() and (lse == -math.inf).all()
    assert fb.last_device_error() == 0


def test_append_takes_a_position_out_of_range_as_zero():
    """Row and queries are those of position 0, and the error word says so; a slot past the cache leaves no row."""
    g = gen(31)
    w, rope = 1.0 + normal(g, C, std=0.2, dtype=torch.float32), rope_table(4)
    kv, q = normal(g, 3, C + R), normal(g, 3, 9, DN + R)
    slots = torch.tensor([5, 17, 32], device="cuda")
    got = []
    for pos in ([0, 0, 3], [4, -1, 3]):
        cache = torch.full((2, 16, C + R), 7.0, dtype=torch.bfloat16, device="cuda")
        qn, qp = fb.mla_append(kv, w, rope, torch.tensor(pos, device="cuda"), slots, cache, q=q)
        assert fb.last_device_error() == 0x100          # the third token's slot, then the positions too
        got.append((cache, qn, qp))
        rows = cache.view(-1, C + R)
        assert sorted((rows != 7).any(-1).nonzero()[:, 0].tolist()) == [5, 17]
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_attention_bad_values_reach_every_row_of_their_request():
    """A NaN key makes all its request's outputs NaN. An infinite entry makes a score +-Inf (or NaN for a zero query
    column), hence a weight NaN or 0: 0 * Inf in that column, at least. The other requests keep their bits."""
    a = make_attention(4, 16, 200, [40, 50, 60, 70], 16, 10)
    clean = call_attention(a)
    rows = a["cache"].view(-1, C + R)
    rows[a["keys_o"][1][7]] = math.nan
    rows[a["keys_o"][2][9], 3] = math.inf
    lse = torch.zeros((4, 16), device="cuda")
    out = call_attention(a, lse)
    assert out[1].isnan().all()
    assert not out[2][:, 3].isfinite().any()
    assert lse[1].isnan().all()
    for b in (0, 3):
        assert torch.equal(out[b].view(torch.int16), clean[b].view(torch.int16)) and lse[b].isfinite().all()


def test_attention_bad_values_in_one_part_of_a_long_row():
    """The same where the row's keys are cut into parts that are joined: one NaN key among 9000, heads of 128 and of 5."""
    for H in (5, 128):
        a = make_attention(2, H, 0, [9000, 3000], 64, 33)
        a["cache"].view(-1, C + R)[a["keys_o"][0][8191]] = math.nan
        lse = torch.zeros((2, H), device="cuda")
        out = call_attention(a, lse)
        assert out[0].isnan().all() and lse[0].isnan().all()
        check_attention(a, out, lse, requests=[1])
    assert fb.last_device_error() == 0


@pytest.mark.parametrize("H,P,own", [(16, 0, 200001), (128, 140003, 60000), (5, 170000, 33)])
def test_attention_of_long_contexts(H, P, own):
    """Hundreds of thousands of keys for one row (several requests' worth of parts); the weights' rounding errors stay
    independent, so the norm's bound is the short rows'."""
    a = make_attention(2, H, P, [own, 7], 64, 41)
    lse = torch.empty((2, H), device="cuda")
    out = call_attention(a, lse)
    check_attention(a, out, lse)
    assert torch.equal(call_attention(a).view(torch.int16), out.view(torch.int16)) and fb.last_device_error() == 0
