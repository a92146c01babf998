"""A small decoder with a mixture of experts on the feed-forward operators, end to end:

    python examples/moe_decoder.py

Every norm adds the residual on the way (awq_rms_norm). Prompts go through projections in 8 bits,
whose rows the norm writes as codes (awq_gemm_i8), new tokens through W4A16 layers of the same
weights; each feed-forward half is a router and its experts (awq_moe_route, awq_moe). The last
tokens of the prompts are decoded again one by one, on the caches that the prompts filled.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_only_w4a16_amd import awq, block, int8, moe  # noqa: E402

F16 = torch.float16


class Linear:
    """The same weights in 4 bits for single tokens and in 8 bits for prompts."""

    def __init__(self, n, k, gen, device):
        w = (torch.randn(n, k, generator=gen) * k ** -0.5).to(F16).to(device)
        self.few, self.many = awq.QuantLinear.from_weight(w), int8.Int8Linear.from_weight(w)

    def __call__(self, x, prompt):
        """x: float16 rows, or (codes, scales) for prompts."""
        if not prompt:
            return self.few(x)
        return self.many(*x) if isinstance(x, tuple) else self.many(x)


class Layer:
    def __init__(self, hidden, ffn, experts, k, heads, kv_heads, head_dim, page, pages, gen, device):
        def rand(*shape, gain):
            return (torch.randn(*shape, generator=gen) * gain).to(F16).to(device)

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.norms = [(1.0 + 0.1 * torch.randn(hidden, generator=gen)).to(F16).to(device) for _ in range(2)]
        self.qkv = Linear((heads + 2 * kv_heads) * head_dim, hidden, gen, device)
        self.o = Linear(hidden, heads * head_dim, gen, device)
        self.moe = moe.MoeLayer.from_weights(
            rand(experts, hidden, gain=2.0 * hidden ** -0.5), rand(experts, ffn, hidden, gain=hidden ** -0.5),
            rand(experts, ffn, hidden, gain=hidden ** -0.5), rand(experts, hidden, ffn, gain=ffn ** -0.5), k)
        self.k_cache = torch.zeros(pages, kv_heads, page, head_dim, dtype=F16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)

    def __call__(self, x, h, positions, inv_freq, slots, attend, prompt):
        """x [tokens, hidden] is the output of the layer before, h the stream that it is added to
        (None: x itself). Returns (this layer's output, the stream)."""
        tokens = x.shape[0]
        n = int8.awq_rms_norm(x, self.norms[0], residual=h, y16=not prompt, i8=prompt)
        h = x if h is None else n.h
        qkv = self.qkv((n.q, n.scale) if prompt else n.y, prompt).view(tokens, -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        q, k = block.awq_rope(q, positions, inv_freq, k=k, v=v, k_cache=self.k_cache, v_cache=self.v_cache,
                              slots=slots, k_out=k_out)
        a = attend(self, q, k, v).reshape(tokens, -1)
        n = int8.awq_rms_norm(self.o(a, prompt), self.norms[1], residual=h)
        return self.moe(n.y), n.h


class Decoder:
    def __init__(self, layers=2, hidden=512, ffn=256, experts=8, k=2, heads=8, kv_heads=2, head_dim=64, page=16,
                 pages=32, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.layers = [Layer(hidden, ffn, experts, k, heads, kv_heads, head_dim, page, pages, gen, device)
                       for _ in range(layers)]
        self.norm = torch.ones(hidden, dtype=F16, device=device)
        self.page, self.device, self.hidden = page, device, hidden
        self.inv_freq, _ = block.rope_frequencies(head_dim, device=device)

    def i32(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def run(self, x, seq, at, table, attend, prompt):
        positions = self.i32(at)
        slots = torch.tensor([table[s][p // self.page] * self.page + p % self.page for s, p in zip(seq, at)],
                             dtype=torch.int64, device=self.device)
        h = None
        for layer in self.layers:
            x, h = layer(x, h, positions, self.inv_freq, slots, attend, prompt)
        return int8.awq_rms_norm(x, self.norm, residual=h).y

    def prefill(self, x, lengths, table, eight_bits=True):
        cu = self.i32([sum(lengths[:i]) for i in range(len(lengths) + 1)])
        seq = [s for s, n in enumerate(lengths) for _ in range(n)]
        at = [p for n in lengths for p in range(n)]
        return self.run(x, seq, at, table, lambda layer, q, k, v: block.awq_attn_prompt(q, k, v, cu), eight_bits)

    def step(self, x, context, table):
        """One new token of each sequence behind `context` positions."""
        cu, ctx = self.i32(list(range(len(context) + 1))), self.i32(context)
        width = max(len(t) for t in table)
        blocks = self.i32([t + [0] * (width - len(t)) for t in table])
        return self.run(x, list(range(len(context))), context, table,
                        lambda layer, q, k, v: block.awq_attn_tree(q, layer.k_cache, layer.v_cache, blocks, ctx, cu, 1),
                        False)


def run(lengths=(37, 5, 64), seed=0, device="cuda"):
    """The prompts' outputs with 8-bit and with W4A16 projections, and each prompt's last token decoded
    behind the others of it."""
    model = Decoder(seed=seed, device=device)
    gen = torch.Generator().manual_seed(seed + 1)
    order = torch.randperm(32, generator=gen).tolist()
    table = [[order.pop() for _ in range(n // model.page + 1)] for n in lengths]
    x = torch.randn(sum(lengths), model.hidden, generator=gen).to(F16).to(device)
    eight = model.prefill(x, list(lengths), table)
    four = model.prefill(x, list(lengths), table, eight_bits=False)
    last = torch.tensor([sum(lengths[:i + 1]) - 1 for i in range(len(lengths))], device=device)
    return eight, four, four[last], model.step(x[last], [n - 1 for n in lengths], table)


if __name__ == "__main__":
    eight, four, want, got = run()
    print(f"last tokens decoded alone against the prompt's pass: largest difference "
          f"{float((want.float() - got.float()).abs().max()):.2e}; 8-bit against 4-bit projections, relative "
          f"{float((eight.float() - four.float()).norm() / four.float().norm()):.2e}")
