"""A small decoder on the quantized layers and the operators around them, end to end:

    python examples/decoder_blocks.py

Prompts of different lengths are packed and prefilled (awq_rope writes keys and values into a
paged cache, awq_attn_prompt attends), then a tree of drafted tokens per sequence is run in
one pass (awq_attn_tree), and the path to one leaf of each tree is decoded again token by
token: the two must agree. Random weights; every projection is a W4A16 layer whose bias,
activation, gate or residual is part of the product (awq_gemm_fused).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_only_w4a16_amd import awq, block  # noqa: E402

F16 = torch.float16


def rms_norm(x):
    xf = x.float()
    return (xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class Cache:
    """Pages of keys and values of one layer, [pages, kv_heads, page, head_dim] each."""

    def __init__(self, pages, kv_heads, page, head_dim, device):
        self.k = torch.zeros(pages, kv_heads, page, head_dim, dtype=F16, device=device)
        self.v = torch.zeros_like(self.k)


class Layer:
    def __init__(self, hidden, ffn, heads, kv_heads, head_dim, gen, device):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim

        def linear(n, k):
            w = (torch.randn(n, k, generator=gen) * k ** -0.5).to(F16).to(device)
            return awq.QuantLinear.from_weight(w, torch.randn(32, k, generator=gen).to(F16).to(device))

        self.qkv = linear((heads + 2 * kv_heads) * head_dim, hidden)
        self.qkv_bias = (0.1 * torch.randn(self.qkv.n, generator=gen)).to(F16).to(device)
        self.o, self.up, self.gate = linear(hidden, heads * head_dim), linear(ffn, hidden), linear(ffn, hidden)
        self.down = linear(hidden, ffn)

    def __call__(self, h, positions, inv_freq, cache, slots, attend):
        """h [tokens, hidden] -> [tokens, hidden]; attend(q, k, v) is the attention."""
        tokens = h.shape[0]
        qkv = self.qkv(rms_norm(h), bias=self.qkv_bias).view(tokens, -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        q, k = block.awq_rope(q, positions, inv_freq, k=k, v=v, k_cache=cache.k, v_cache=cache.v, slots=slots,
                              k_out=k_out)
        a = attend(q, k, v)
        h = self.o(a.reshape(tokens, -1), residual=h)
        x = rms_norm(h)
        return self.down(self.gate(x, act="silu", mul=self.up(x)), residual=h)


class Decoder:
    def __init__(self, layers=2, hidden=512, ffn=1024, heads=8, kv_heads=2, head_dim=64, page=16, pages=64, seed=0,
                 device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.layers = [Layer(hidden, ffn, heads, kv_heads, head_dim, gen, device) for _ in range(layers)]
        self.caches = [Cache(pages, kv_heads, page, head_dim, device) for _ in range(layers)]
        self.page, self.device = page, device
        self.inv_freq, _ = block.rope_frequencies(head_dim, device=device)

    def i32(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def slots(self, table, seq, at):
        """Cache slots of positions `at` of the sequences `seq` (lists of one length)."""
        return torch.tensor([table[s][p // self.page] * self.page + p % self.page for s, p in zip(seq, at)],
                            dtype=torch.int64, device=self.device)

    def prefill(self, h, lengths, table):
        """h: the packed prompts' embeddings."""
        cu = self.i32([sum(lengths[:i]) for i in range(len(lengths) + 1)])
        seq = [s for s, n in enumerate(lengths) for _ in range(n)]
        at = [p for n in lengths for p in range(n)]
        positions, slots = self.i32(at), self.slots(table, seq, at)
        for layer, cache in zip(self.layers, self.caches):
            h = layer(h, positions, self.inv_freq, cache, slots, lambda q, k, v: block.awq_attn_prompt(q, k, v, cu))
        return h

    def step(self, h, context, parents, table):
        """New tokens behind `context` cached positions of each sequence; parents[s][t] is the
        index of new token t's parent among them, or -1 (one token: plain decoding)."""
        counts = [len(p) for p in parents]
        depth = []
        for p in parents:
            d = []
            for t in p:
                d.append(0 if t < 0 else d[t] + 1)
            depth.append(d)
        seq = [s for s, n in enumerate(counts) for _ in range(n)]
        positions = self.i32([context[s] + x for s, d in enumerate(depth) for x in d])
        slots = self.slots(table, seq, [context[s] + t for s, n in enumerate(counts) for t in range(n)])
        mask = torch.cat([block.tree_mask(p) for p in parents]).to(self.device)
        cu = self.i32([sum(counts[:i]) for i in range(len(counts) + 1)])
        width = max(len(t) for t in table)
        blocks, ctx = self.i32([t + [0] * (width - len(t)) for t in table]), self.i32(context)
        for layer, cache in zip(self.layers, self.caches):
            h = layer(h, positions, self.inv_freq, cache, slots,
                      lambda q, k, v: block.awq_attn_tree(q, cache.k, cache.v, blocks, ctx, cu, max(counts), mask=mask))
        return h


def run(lengths=(37, 5, 64), seed=0, device="cuda"):
    """(largest difference, largest value) between a tree's pass and decoding one path of it
    token by token."""
    model = Decoder(seed=seed, device=device)
    gen = torch.Generator().manual_seed(seed + 1)
    hidden = model.layers[0].o.n

    def embed(n):
        return torch.randn(n, hidden, generator=gen).to(F16).to(device)

    order = torch.randperm(60, generator=gen).tolist()
    table = [[order.pop() for _ in range((n + 16) // model.page + 1)] for n in lengths]
    model.prefill(embed(sum(lengths)), list(lengths), table)
    trees = [[-1, 0, 0, 1, 2, 4], [-1, -1, 1, 1, 3], [-1, 0, 1, 2, 0, 4, 4]]
    paths = [[0, 2, 4, 5], [1, 3, 4], [0, 4, 6]]
    drafts = [embed(len(t)) for t in trees]
    out = model.step(torch.cat(drafts), list(lengths), trees, table)
    diff = top = 0.0
    at = 0
    for s, path in enumerate(paths):
        for i, token in enumerate(path):   # one sequence at a time, one token at a time
            h = model.step(drafts[s][token:token + 1], [lengths[s] + i], [[-1]], [table[s]])
            tree = out[at + token]
            diff = max(diff, float((h[0].float() - tree.float()).abs().max()))
            top = max(top, float(tree.float().abs().max()))
        at += len(trees[s])
    return diff, top


if __name__ == "__main__":
    difference, largest = run()
    print(f"tree pass against token-by-token decoding: largest difference {difference:.2e}, "
          f"largest value {largest:.2f}")
