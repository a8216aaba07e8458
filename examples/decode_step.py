"""A decode loop of one MLA + MoE transformer layer over a paged latent cache.

A prompt that all requests share is written into the cache once; then every step takes one token per request:

    q, kv = FP8 linears of the normed hidden state
    mla_append     the latent normed, its key part and the queries rotated, the token's cache row written
    mla_absorb     q_nope into the latent space ("qk")
    mla_attention  the request's token against the shared prompt and the request's own keys
    mla_absorb     the latent output into the heads' values ("v"), then the output linear
    moe_layer      gate, routed and shared experts of the step's tokens (at most 32) in one kernel

    python examples/decode_step.py [--batch 4] [--prefix 300] [--steps 5] [--graph]

prints each step's hidden state norm and how far the attention is from its formula in 64 bits. With --graph one step
is captured once and replayed: lengths, positions and slots are device tensors, so nothing in it depends on the host.
Weights and inputs are random; the sizes are a small layer's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_quant_gb300 as fb  # noqa: E402

LATENT, ROPE, NOPE, VALUE = fb.MLA_LATENT, fb.MLA_ROPE, fb.MLA_NOPE, 128


def rms_norm(x, w, eps=1e-6):
    h = x.float()
    return (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * w).to(torch.bfloat16)


def rope_table(n, device, base=10000.0):
    """[n, 32, 2]: cosine and sine of position * base^(-2 i / 64)."""
    inv = base ** (-torch.arange(0, ROPE, 2, device=device, dtype=torch.float64) / ROPE)
    a = torch.arange(n, device=device, dtype=torch.float64)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


class Layer:
    """One layer's weights: FP8 linears with block scales, the gate in bf16, norms in fp32."""

    def __init__(self, dim=1024, heads=16, experts=32, inter=512, topk=4, shared=1, max_pos=4096, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def fp8(rows, cols):
            return fb.weight_quant(torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5)

        self.dim, self.heads, self.topk, self.shared = dim, heads, topk, shared
        self.norm_attn = torch.ones(dim, device=device)
        self.norm_ffn = torch.ones(dim, device=device)
        self.norm_kv = torch.ones(LATENT, device=device)
        self.wq = fp8(heads * (NOPE + ROPE), dim)
        self.wkv_a = fp8(LATENT + ROPE, dim)
        self.wkv_b = fp8(heads * (NOPE + VALUE), LATENT)
        self.wo = fp8(dim, heads * VALUE)
        self.gate = (torch.randn(experts, dim, generator=g, device=device) * dim ** -0.5).to(torch.bfloat16)
        n = experts + shared
        self.w1, self.w3, self.w2 = fp8(n * inter, dim), fp8(n * inter, dim), fp8(n * dim, inter)
        self.rope = rope_table(max_pos, device)
        self.scale = (NOPE + ROPE) ** -0.5


class Cache:
    """Pages of latent rows: the prompt's, shared, and each request's own."""

    def __init__(self, batch, prefix, own, page=64, device="cuda"):
        pre, each = -(-prefix // page), -(-own // page)
        self.page, self.prefix = page, prefix
        self.rows = torch.zeros(pre + batch * each, page, LATENT + ROPE, dtype=torch.bfloat16, device=device)
        ids = torch.randperm(pre + batch * each, device=device).to(torch.int32)
        self.prefix_pages = ids[:pre].contiguous()
        self.table = ids[pre:].view(batch, each).contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)

    def slots(self):
        """The row that each request's next token goes to."""
        at = self.lens.long()
        pages = self.table.gather(1, (at // self.page)[:, None]).squeeze(1).long()
        return pages * self.page + at % self.page

    def prefix_slots(self):
        j = torch.arange(self.prefix, device=self.rows.device)
        return self.prefix_pages[j // self.page].long() * self.page + j % self.page


def write_prompt(layer, cache, x):
    """The prompt's rows, once: x bf16 [prefix, dim]."""
    kv = fb.linear(rms_norm(x, layer.norm_attn), *layer.wkv_a)
    pos = torch.arange(x.shape[0], device=x.device)
    fb.mla_append(kv, layer.norm_kv, layer.rope, pos, cache.prefix_slots(), cache.rows)


def step(layer, cache, x):
    """One token per request: x bf16 [batch, dim] -> the layer's output and the attention's operands and output."""
    b = x.shape[0]
    h = rms_norm(x, layer.norm_attn)
    q = fb.linear(h, *layer.wq).view(b, layer.heads, NOPE + ROPE)
    kv = fb.linear(h, *layer.wkv_a)
    q_nope, q_pe = fb.mla_append(kv, layer.norm_kv, layer.rope, cache.prefix + cache.lens.long(), cache.slots(),
                                 cache.rows, q=q)
    cache.lens += 1
    q_lat = fb.mla_absorb(q_nope, *layer.wkv_b, "qk")
    o = fb.mla_attention(q_lat, q_pe, cache.rows, cache.table, cache.lens, layer.scale,
                         prefix_pages=cache.prefix_pages, prefix_len=cache.prefix)
    v = fb.mla_absorb(o, *layer.wkv_b, "v")
    x = x + fb.linear(v.view(b, layer.heads * VALUE), *layer.wo)
    y = fb.moe_layer(rms_norm(x, layer.norm_ffn), layer.gate, *layer.w1, *layer.w3, *layer.w2, layer.topk,
                     n_shared=layer.shared)
    return x + y, q_lat, q_pe, o


def attention_formula(layer, cache, q_lat, q_pe):
    """softmax(scale <[q_lat, q_pe], c>) c[0:512] in 64 bits, request by request."""
    rows = cache.rows.view(-1, LATENT + ROPE)
    out = torch.empty(q_lat.shape, dtype=torch.float64, device=q_lat.device)
    shared = rows[cache.prefix_slots()].double()
    for b, n in enumerate(cache.lens.tolist()):
        j = torch.arange(n, device=rows.device)
        own = rows[cache.table[b][j // cache.page].long() * cache.page + j % cache.page].double()
        c = torch.cat((shared, own))
        s = torch.cat((q_lat[b], q_pe[b]), -1).double() @ c.T * layer.scale
        out[b] = torch.softmax(s, -1) @ c[:, :LATENT]
    return out


def main(argv=None):
    a = argparse.ArgumentParser(description="decode steps of one MLA + MoE layer")
    a.add_argument("--batch", type=int, default=4)
    a.add_argument("--prefix", type=int, default=300)
    a.add_argument("--steps", type=int, default=5)
    a.add_argument("--graph", action="store_true")
    a = a.parse_args(argv)
    if not 1 <= a.batch <= fb.MOE_LAYER_MAX_TOKENS:
        raise SystemExit(f"--batch: 1 to {fb.MOE_LAYER_MAX_TOKENS}")
    layer, cache = Layer(), Cache(a.batch, a.prefix, a.steps + 2)
    g = torch.Generator(device="cuda").manual_seed(1)
    write_prompt(layer, cache, torch.randn(a.prefix, layer.dim, generator=g, device="cuda").to(torch.bfloat16))
    first = torch.randn(a.batch, layer.dim, generator=g, device="cuda").to(torch.bfloat16)
    x, graph, seen = first.clone(), None, []
    if a.graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())  # weights, page table, lengths and prompt are written there
        with torch.cuda.stream(side):
            step(layer, cache, x)  # workspaces of this stream
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs = step(layer, cache, x)
                x.copy_(outs[0])
        torch.cuda.current_stream().wait_stream(side)
        cache.lens.zero_()
        x.copy_(first)
    for i in range(a.steps):
        if graph is not None:
            graph.replay()
        else:
            outs = step(layer, cache, x)
            x = outs[0]
        want = attention_formula(layer, cache, outs[1], outs[2])
        off = ((outs[3].double() - want).norm() / want.norm()).item()
        norm = x.float().norm().item()
        seen.append((norm, off))
        print(f"step {i}: |x| = {norm:.4f}, attention off its formula by {off:.2e}")
    if fb.last_device_error():
        raise SystemExit(f"device error {fb.last_device_error():#x}")
    return seen


if __name__ == "__main__":
    main()
