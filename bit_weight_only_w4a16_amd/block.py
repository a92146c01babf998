"""Binding of the decoder-block operators (``awq_block.h``) around the quantized products.

Same manner as ``awq``: each function has the name of its C entry point, checks device,
dtype, layout and extents, allocates outputs with PyTorch, runs on PyTorch's current stream
and raises ``AwqError`` on a non-zero status. Operands may be strided views whose last
dimension is contiguous (slices of one fused projection, a cache with its heads or its
slots outermost).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import awq

DT = {torch.float16: 0, torch.bfloat16: 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
TREE_MAX_TOKENS = 64

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_f32 = ctypes.c_float


class RopeArgs(ctypes.Structure):
    """awq_rope_args of awq_block.h."""
    _fields_ = ([(n, _vp) for n in ("q", "q_out", "k", "k_out", "v", "k_cache", "v_cache", "positions",
                                    "inv_freq", "slots")]
                + [(n, _i64) for n in ("tokens", "q_token", "q_head", "qo_token", "qo_head", "k_token", "k_head",
                                       "ko_token", "ko_head", "v_token", "v_head", "cache_page", "cache_head",
                                       "cache_slot", "pages")]
                + [(n, _i32) for n in ("page_size", "q_heads", "kv_heads", "head_dim", "rot_dim", "dtype",
                                       "interleaved", "inverse")]
                + [("scale", _f32), ("reserved", _i32)])


class AttnPromptArgs(ctypes.Structure):
    """awq_attn_prompt_args of awq_block.h."""
    _fields_ = ([(n, _vp) for n in ("q", "k", "v", "out", "cu")]
                + [(n, _i64) for n in ("tokens", "seqs", "q_token", "q_head", "k_token", "k_head", "v_token",
                                       "v_head", "o_token", "o_head")]
                + [(n, _i32) for n in ("q_heads", "kv_heads", "head_dim", "dtype")]
                + [("scale", _f32), ("reserved", _i32)])


class AttnTreeArgs(ctypes.Structure):
    """awq_attn_tree_args of awq_block.h."""
    _fields_ = ([(n, _vp) for n in ("q", "k_cache", "v_cache", "out", "block_table", "ctx_lens", "cu_q", "mask",
                                    "ws")]
                + [("ws_bytes", ctypes.c_size_t)]
                + [(n, _i64) for n in ("tokens", "seqs", "table_width", "pages", "q_token", "q_head", "o_token",
                                       "o_head", "cache_page", "cache_head", "cache_slot")]
                + [(n, _i32) for n in ("page_size", "max_q", "q_heads", "kv_heads", "head_dim", "dtype")]
                + [("scale", _f32), ("reserved", _i32)])


class Epilogue(ctypes.Structure):
    """awq_epilogue of awq_block.h."""
    _fields_ = [("bias", _vp), ("mul", _vp), ("residual", _vp), ("act", _i32), ("reserved", _i32)]


_SIGNATURES = {
    "awq_gemm_fused": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp, ctypes.c_size_t,
                                      _vp]),
    "awq_rope": (ctypes.c_int, [_vp, _vp]),
    "awq_attn_prompt": (ctypes.c_int, [_vp, _vp]),
    "awq_attn_tree_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, _i32, _i32, _i32, _i32, _i32]),
    "awq_attn_tree": (ctypes.c_int, [_vp, _vp]),
}
EXPORTS = tuple(_SIGNATURES)

_lib = None


def lib() -> ctypes.CDLL:
    """The library of ``awq`` with this module's entry points declared."""
    global _lib
    if _lib is None:
        handle = awq.lib()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _heads(t, name: str, dtype=None) -> None:
    """A packed operand [tokens, heads, D] of 16-bit elements with contiguous heads."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in DT or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'float16 or bfloat16'}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if t.stride(2) != 1:
        raise ValueError(f"the elements of a head of {name} must be contiguous")


def _strides(t) -> tuple:
    """(token, head) strides; a dimension of one has none that matters."""
    st, sh, _ = t.stride()
    n, h, d = t.shape
    return (st if n > 1 else max(st, h * d), sh if h > 1 else d)


def _cache(k_cache, v_cache, dtype, heads: int, d: int, device) -> tuple:
    """Checks a paged cache [pages, kv_heads, page_size, D] and returns its strides."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or t.device != device:
            raise ValueError(f"{name} must be a tensor on {device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != 4 or t.shape[1] != heads or t.shape[3] != d:
            raise ValueError(f"{name} must be [pages, {heads}, page_size, {d}], got {tuple(t.shape)}")
        if t.stride(3) != 1:
            raise ValueError(f"the elements of a slot of {name} must be contiguous")
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must have one shape and one layout")
    sp, sh, ss, _ = k_cache.stride()
    return sp, sh, max(ss, d) if k_cache.shape[2] == 1 else ss


def _like(out, name: str, ref: torch.Tensor) -> torch.Tensor:
    if out is None:
        return torch.empty(ref.shape, dtype=ref.dtype, device=ref.device)
    _heads(out, name, ref.dtype)
    awq._shape(out, name, ref.shape)
    awq._same_device(ref, **{name: out})
    return out


def awq_gemm_fused(x, inv_s_c, packed, n: int, k: int, group: int = awq.GROUP, fmt: int = awq.FMT_ASYM, *,
                   bias=None, act: str = "none", mul=None, residual=None, y=None, ws=None) -> torch.Tensor:
    """awq_gemm with an element-wise tail, y = act(x . W^T + bias) * mul + residual, rounded
    once: bias fp16 [N], mul and residual fp16 [M, N], act one of ACTS. y may be mul or
    residual itself."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {tuple(ACTS)}")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be [M, K]")
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float16, device=x.device)
    awq._shape(y, "y", (m, n))
    awq._shape(inv_s_c, "inv_s_c", (k,))
    awq._shape(bias, "bias", (n,))
    awq._shape(mul, "mul", (m, n))
    awq._shape(residual, "residual", (m, n))
    awq._at_least(packed, "packed", awq.awq_repacked_bytes(n, k, group, fmt))
    awq._same_device(x, inv_s_c=inv_s_c, packed=packed, bias=bias, mul=mul, residual=residual, y=y, ws=ws)
    f16 = torch.float16
    tail = Epilogue(awq._opt(bias, "bias", f16), awq._opt(mul, "mul", f16), awq._opt(residual, "residual", f16),
                    ACTS[act], 0)
    awq._check(lib().awq_gemm_fused(awq._dev(x, "x", f16), awq._opt(inv_s_c, "inv_s_c", f16),
                                    awq._dev(packed, "packed", torch.uint8), m, n, k, group, fmt,
                                    ctypes.byref(tail), awq._dev(y, "y", f16), awq._opt(ws, "ws", torch.uint8),
                                    0 if ws is None else ws.numel(), awq._stream(x.device)), "awq_gemm_fused")
    return y


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: int = 8192, low: float = 1.0, high: float = 4.0, device="cpu"):
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
    if q is None and k is None:
        raise ValueError("q or k is required")
    ref = q if q is not None else k
    _heads(ref, "q" if q is not None else "k")
    dtype, device, (tokens, _, d) = ref.dtype, ref.device, ref.shape
    args = RopeArgs(tokens=tokens, head_dim=d, rot_dim=2 * inv_freq.numel(), dtype=DT[dtype],
                    interleaved=int(interleaved), inverse=int(inverse), scale=scale)
    if 2 * inv_freq.numel() > d:
        raise ValueError("inv_freq has more pairs than the head")
    args.positions = awq._dev(positions, "positions", torch.int32)
    args.inv_freq = awq._dev(inv_freq, "inv_freq", torch.float32)
    awq._shape(positions, "positions", (tokens,))
    awq._same_device(ref, positions=positions, inv_freq=inv_freq, slots=slots)
    if q is not None:
        q_out = _like(q_out, "q_out", q)
        args.q, args.q_out, args.q_heads = q.data_ptr(), q_out.data_ptr(), q.shape[1]
        args.q_token, args.q_head = _strides(q)
        args.qo_token, args.qo_head = _strides(q_out)
    if k is not None:
        _heads(k, "k", dtype)
        if k.shape[0] != tokens or k.shape[2] != d:
            raise ValueError("k must have q's tokens and head size")
        awq._same_device(ref, k=k)
        args.k, args.kv_heads = k.data_ptr(), k.shape[1]
        args.k_token, args.k_head = _strides(k)
        if k_cache is None or k_out is not None:
            k_out = _like(k_out, "k_out", k)
            args.k_out = k_out.data_ptr()
            args.ko_token, args.ko_head = _strides(k_out)
        if (k_cache is None) != (v_cache is None):
            raise ValueError("k_cache and v_cache go together")
        if k_cache is not None:
            if v is None or slots is None:
                raise ValueError("a cache needs v and slots")
            _heads(v, "v", dtype)
            awq._shape(v, "v", k.shape)
            awq._shape(slots, "slots", (tokens,))
            awq._same_device(ref, v=v)
            args.cache_page, args.cache_head, args.cache_slot = _cache(k_cache, v_cache, dtype, k.shape[1], d, device)
            args.pages, args.page_size = k_cache.shape[0], k_cache.shape[2]
            args.k_cache, args.v_cache, args.v = k_cache.data_ptr(), v_cache.data_ptr(), v.data_ptr()
            args.v_token, args.v_head = _strides(v)
            args.slots = awq._dev(slots, "slots", torch.int64)
    elif k_cache is not None or v_cache is not None or k_out is not None:
        raise ValueError("a cache or k_out needs k")
    awq._check(lib().awq_rope(ctypes.byref(args), awq._stream(device)), "awq_rope")
    return q_out, k_out


def awq_attn_prompt(q, k, v, cu_seqlens, scale: float | None = None, out=None) -> torch.Tensor:
    """Causal attention of packed prompts: q [tokens, q_heads, D], k and v [tokens, kv_heads,
    D]; sequence b is the tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32 [seqs + 1]).
    scale defaults to D ** -0.5. Tokens in no sequence are not written."""
    _heads(q, "q")
    _heads(k, "k", q.dtype)
    _heads(v, "v", q.dtype)
    tokens, hq, d = q.shape
    hkv = k.shape[1]
    awq._shape(k, "k", (tokens, hkv, d))
    awq._shape(v, "v", (tokens, hkv, d))
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [seqs + 1]")
    out = _like(out, "out", q)
    awq._same_device(q, k=k, v=v, cu_seqlens=cu_seqlens)
    args = AttnPromptArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                          awq._dev(cu_seqlens, "cu_seqlens", torch.int32), tokens, cu_seqlens.numel() - 1,
                          *_strides(q), *_strides(k), *_strides(v), *_strides(out), hq, hkv, d, DT[q.dtype],
                          d ** -0.5 if scale is None else scale, 0)
    awq._check(lib().awq_attn_prompt(ctypes.byref(args), awq._stream(q.device)), "awq_attn_prompt")
    return out


def awq_attn_tree_workspace_bytes(tokens: int, seqs: int, table_width: int, page_size: int, max_q: int,
                                  q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().awq_attn_tree_workspace_bytes(tokens, seqs, table_width, page_size, max_q, q_heads,
                                                   kv_heads, head_dim))


def awq_attn_tree(q, k_cache, v_cache, block_table, ctx_lens, cu_q, max_q: int, mask=None,
                  scale: float | None = None, out=None, ws=None) -> torch.Tensor:
    """Attention of the new tokens q [tokens, q_heads, D] over a paged cache [pages, kv_heads,
    page_size, D] that already holds their keys and values behind each sequence's context.
    block_table int32 [seqs, width], ctx_lens int32 [seqs], cu_q int32 [seqs + 1], max_q the
    most new tokens of a sequence (<= 64). mask int64 [tokens]: bit j of a token's word lets
    it see new token j of its sequence (`tree_mask` forms it from a tree); without one, new
    tokens see those up to themselves. A token that sees nothing gets zeros."""
    _heads(q, "q")
    tokens, hq, d = q.shape
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, D]")
    pages, hkv, page_size, _ = k_cache.shape
    cache = _cache(k_cache, v_cache, q.dtype, hkv, d, q.device)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [seqs, width]")
    seqs, width = block_table.shape
    awq._shape(ctx_lens, "ctx_lens", (seqs,))
    awq._shape(cu_q, "cu_q", (seqs + 1,))
    awq._shape(mask, "mask", (tokens,))
    out = _like(out, "out", q)
    awq._same_device(q, block_table=block_table, ctx_lens=ctx_lens, cu_q=cu_q, mask=mask, ws=ws)
    if ws is None:
        ws = _workspace(awq_attn_tree_workspace_bytes(tokens, seqs, width, page_size, max_q, hq, hkv, d), q.device)
    args = AttnTreeArgs(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                        awq._dev(block_table, "block_table", torch.int32),
                        awq._dev(ctx_lens, "ctx_lens", torch.int32), awq._dev(cu_q, "cu_q", torch.int32),
                        awq._opt(mask, "mask", torch.int64), awq._opt(ws, "ws", torch.uint8),
                        0 if ws is None else ws.numel(), tokens, seqs, width, pages, *_strides(q), *_strides(out),
                        *cache, page_size, max_q, hq, hkv, d, DT[q.dtype], d ** -0.5 if scale is None else scale, 0)
    awq._check(lib().awq_attn_tree(ctypes.byref(args), awq._stream(q.device)), "awq_attn_tree")
    return out


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


_WS = {}


def _workspace(need: int, device) -> torch.Tensor | None:
    """A workspace of at least `need` bytes, cached per device and stream and grown on
    demand, as awq.workspace."""
    if need == 0:
        return None
    key = (device.index, awq._stream(device))
    cur = _WS.get(key)
    if cur is None or cur.numel() < need:
        cur = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=device)
        _WS[key] = cur
    return cur
