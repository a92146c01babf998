"""The decoder-block operators (``awq_block.h``) around the quantized products.

Same manner as ``awq``: each function has the name of its C entry point, checks device,
dtype, layout and extents, allocates outputs with PyTorch, runs on PyTorch's current stream
and raises ``AwqError`` on a non-zero status. The checks and the marshalling are in the
extension module ``_block`` (``csrc/binding.cpp``); if it is not built, the import raises.
Operands may be strided views whose last dimension is contiguous (slices of one fused
projection, a cache with its heads or its slots outermost).
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import awq

try:
    from . import _block
except ImportError as e:
    raise ImportError(f"the extension module of {__name__} does not load ({e}); run "
                      "`python -m bit_weight_only_w4a16_amd.build`") from e

DT = {torch.float16: 0, torch.bfloat16: 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
TREE_MAX_TOKENS = 64
EXPORTS = ("awq_attn_prompt", "awq_attn_tree", "awq_attn_tree_workspace_bytes", "awq_gemm_fused", "awq_rope")

_block.setup(awq._stream, awq.scratch, awq.AwqError)


def awq_gemm_fused(x, inv_s_c, packed, n: int, k: int, group: int = awq.GROUP, fmt: int = awq.FMT_ASYM, *,
                   bias=None, act: str = "none", mul=None, residual=None, y=None, ws=None) -> torch.Tensor:
    """awq_gemm with an element-wise tail, y = act(x . W^T + bias) * mul + residual, rounded
    once: bias fp16 [N], mul and residual fp16 [M, N], act one of ACTS. y may be mul or
    residual itself."""
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {tuple(ACTS)}")
    return _block.gemm_fused(x, inv_s_c, packed, n, k, group, fmt, bias, code, mul, residual, y, ws)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: int = 8192, low: float = 1.0, high: float | None = None, device="cpu"):
    """(inv_freq float32 [rot_dim / 2], scale): base ** (-2 i / rot_dim), stretched for
    contexts `factor` times as long as the `original` one:

      "linear"  every frequency divided by `factor` (positions interpolated);
      "ntk"     the base enlarged to base * factor ** (rot_dim / (rot_dim - 2)): the slowest
                frequency divided by `factor`, the fastest kept;
      "bands"   frequencies that turn fewer than `low` times over `original` divided by
                `factor`, those that turn more than `high` times kept, linear in the turns
                between;
      "yarn"    the same blend, linear in the pair's index between the pairs that turn `high`
                and `low` times, and scale = 0.1 ln(factor) + 1 on q and k.

    `high` is 4 for "bands" and 32 for "yarn" unless given, as published for each.
    Computed once, in float64, and rounded to float32."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim
    freq, scale = base ** -i, 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "ntk":
        if rot_dim == 2:
            raise ValueError("ntk scaling needs more than one pair")
        freq = (base * factor ** (rot_dim / (rot_dim - 2))) ** -i
    elif scaling in ("bands", "yarn"):
        if high is None:
            high = 4.0 if scaling == "bands" else 32.0
        if not 0 < low < high:
            raise ValueError("low must be positive and less than high")
        if scaling == "bands":
            turns = original * freq / (2 * math.pi)
            keep = ((turns - low) / (high - low)).clamp(0, 1)
        else:
            def pair(turns):   # the (fractional) pair that turns so often over `original`
                return rot_dim * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            first = max(math.floor(pair(high)), 0)
            last = min(math.ceil(pair(low)), rot_dim - 1)
            at = torch.arange(rot_dim // 2, dtype=torch.float64)
            keep = 1 - ((at - first) / max(last - first, 1e-3)).clamp(0, 1)
            scale = 0.1 * math.log(factor) + 1.0
        freq = freq / factor * (1 - keep) + freq * keep
    elif scaling is not None:
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(torch.float32).to(device), scale


def awq_rope(q, positions, inv_freq, k=None, v=None, k_cache=None, v_cache=None, slots=None,
             interleaved: bool = False, inverse: bool = False, scale: float = 1.0, q_out=None, k_out=None):
    """Rotate q [tokens, q_heads, D] and k [tokens, kv_heads, D] by positions (int32
    [tokens]) * inv_freq (float32 [rot_dim / 2]). With a cache ([pages, kv_heads, page_size,
    D]) the rotated k and v go to its slots (int64 [tokens], page * page_size + slot;
    negative: not stored). Returns (q_out, k_out); k_out is None where k goes to the cache
    and no k_out is given. q_out may be q itself and k_out k itself."""
    return _block.rope(q, positions, inv_freq, k, v, k_cache, v_cache, slots, interleaved, inverse, scale, q_out,
                       k_out)


def awq_attn_prompt(q, k, v, cu_seqlens, scale: float | None = None, out=None) -> torch.Tensor:
    """Causal attention of packed prompts: q [tokens, q_heads, D], k and v [tokens, kv_heads,
    D]; sequence b is the tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32 [seqs + 1]).
    scale defaults to D ** -0.5. Tokens in no sequence are not written."""
    return _block.attn_prompt(q, k, v, cu_seqlens, scale, out)


@functools.lru_cache(maxsize=4096)
def awq_attn_tree_workspace_bytes(tokens: int, seqs: int, table_width: int, page_size: int, max_q: int,
                                  q_heads: int, kv_heads: int, head_dim: int) -> int:
    fn = awq.lib().awq_attn_tree_workspace_bytes
    fn.restype = ctypes.c_size_t
    fn.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int32] * 5
    return int(fn(tokens, seqs, table_width, page_size, max_q, q_heads, kv_heads, head_dim))


def awq_attn_tree(q, k_cache, v_cache, block_table, ctx_lens, cu_q, max_q: int, mask=None,
                  scale: float | None = None, out=None, ws=None) -> torch.Tensor:
    """Attention of the new tokens q [tokens, q_heads, D] over a paged cache [pages, kv_heads,
    page_size, D] that already holds their keys and values behind each sequence's context.
    block_table int32 [seqs, width], ctx_lens int32 [seqs], cu_q int32 [seqs + 1], max_q the
    most new tokens of a sequence (<= 64). mask int64 [tokens]: bit j of a token's word lets
    it see new token j of its sequence (`tree_mask` forms it from a tree); without one, new
    tokens see those up to themselves. A token that sees nothing gets zeros. ws: uint8,
    awq_attn_tree_workspace_bytes() of them; when absent, one cached per stream and thread or, under
    capture, one of the graph's own (awq.scratch). Graphs captured with the same ws must not be
    replayed side by side."""
    return _block.attn_tree(q, k_cache, v_cache, block_table, ctx_lens, cu_q, max_q, mask, scale, out, ws)


def tree_mask(parents) -> torch.Tensor:
    """int64 [tokens] mask words of one tree: parents[t] is the index of token t's parent
    among the new tokens (less than t), or -1 where it follows the context."""
    words = []
    for t, p in enumerate(parents):
        p = int(p)
        if not -1 <= p < t:
            raise ValueError("a token's parent must stand before it")
        words.append((words[p] if p >= 0 else 0) | 1 << t)
    if len(words) > TREE_MAX_TOKENS:
        raise ValueError(f"at most {TREE_MAX_TOKENS} tokens in a tree")
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)
