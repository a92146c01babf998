"""Binding of the decoder-block operators (``awq_block.h``) around the quantized products.

Same manner as ``awq``: each function has the name of its C entry point, checks device,
dtype, layout and extents, allocates outputs with PyTorch, runs on PyTorch's current stream
and raises ``AwqError`` on a non-zero status. Operands may be strided views whose last
dimension is contiguous (slices of one fused projection, a cache with its heads or its
slots outermost).
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct

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


# The argument structures as the C compiler lays them out, packed in one call: a call's
# arguments are bytes that live as long as the call.
_ROPE = struct.Struct("@10P15q8ifi")
_PROMPT = struct.Struct("@5P10q4ifi")
_TREE = struct.Struct("@9PN11q6ifi")
_EPILOGUE = struct.Struct("@3P2i")


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _refuse(ref, dtype, packed=(), vectors=()) -> None:
    """Says what is wrong with a call's tensors, which the caller found in one test of them
    all: `packed` operands [tokens, heads, D] as (name, tensor), `vectors` as (name, tensor,
    dtype, shape)."""
    for name, t in packed:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a device tensor")
        if t.dtype not in DT or t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype if dtype in DT else 'float16 or bfloat16'}, got {t.dtype}")
        if t.dim() != 3:
            raise ValueError(f"{name} must be [tokens, heads, head_dim]")
        if t.stride(2) != 1:
            raise ValueError(f"the elements of a head of {name} must be contiguous")
        awq._same_device(ref, **{name: t})
    for name, t, want, shape in vectors:
        if t is not None:
            awq._dev(t, name, want)
            awq._shape(t, name, shape)
            awq._same_device(ref, **{name: t})


def _packed(t, dtype, index: int) -> bool:
    """Whether t is a packed operand [tokens, heads, D] of one type on one device."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == 3
            and t.stride(2) == 1)


def _vector(t, dtype, index: int, shape: tuple) -> bool:
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous())


def _strides(t, heads: int, d: int) -> tuple:
    """(token, head) strides; a dimension of one has none that matters."""
    st, sh, _ = t.stride()
    return (st if t.shape[0] > 1 else max(st, heads * d), sh if heads > 1 else d)


def _cache(k_cache, v_cache, dtype, heads: int, d: int, index: int) -> tuple:
    """Checks a paged cache [pages, kv_heads, page_size, D]: (pages, page_size, strides)."""
    if (isinstance(k_cache, torch.Tensor) and isinstance(v_cache, torch.Tensor) and k_cache.dtype is dtype
            and v_cache.dtype is dtype and k_cache.get_device() == index and v_cache.get_device() == index
            and k_cache.dim() == 4):
        shape, strides = k_cache.shape, k_cache.stride()
        pages, h, page_size, width = shape
        if h == heads and width == d and strides[3] == 1 and v_cache.shape == shape and v_cache.stride() == strides:
            return pages, page_size, strides[0], strides[1], strides[2] if page_size > 1 else max(strides[2], d)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or t.get_device() != index:
            raise ValueError(f"{name} must be a tensor on the operands' device")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != 4 or t.shape[1] != heads or t.shape[3] != d:
            raise ValueError(f"{name} must be [pages, {heads}, page_size, {d}], got {tuple(t.shape)}")
        if t.stride(3) != 1:
            raise ValueError(f"the elements of a slot of {name} must be contiguous")
    raise ValueError("k_cache and v_cache must have one shape and one layout")


def _output(out, name: str, ref: torch.Tensor, index: int) -> torch.Tensor:
    if out is None:
        return ref.new_empty(ref.shape)
    if not (_packed(out, ref.dtype, index) and out.shape == ref.shape):
        _refuse(ref, ref.dtype, ((name, out),))
        awq._shape(out, name, ref.shape)
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
    m, index, f16 = x.shape[0], x.get_device(), torch.float16
    if y is None:
        y = x.new_empty((m, n))
    need = awq.awq_repacked_bytes(n, k, group, fmt)
    if not (index >= 0 and _vector(x, f16, index, (m, k)) and _vector(y, f16, index, (m, n))
            and (inv_s_c is None or _vector(inv_s_c, f16, index, (k,)))
            and (bias is None or _vector(bias, f16, index, (n,)))
            and (mul is None or _vector(mul, f16, index, (m, n)))
            and (residual is None or _vector(residual, f16, index, (m, n)))):
        _refuse(x, f16, (), (("x", x, f16, (m, k)), ("y", y, f16, (m, n)), ("inv_s_c", inv_s_c, f16, (k,)),
                             ("bias", bias, f16, (n,)), ("mul", mul, f16, (m, n)),
                             ("residual", residual, f16, (m, n))))
    awq._dev(packed, "packed", torch.uint8)
    awq._at_least(packed, "packed", need)
    ws_bytes = 0
    if ws is not None:
        awq._dev(ws, "ws", torch.uint8)
        ws_bytes = ws.numel()
    if packed.get_device() != index or (ws is not None and ws.get_device() != index):
        awq._same_device(x, packed=packed, ws=ws)
    tail = _EPILOGUE.pack(_ptr(bias), _ptr(mul), _ptr(residual), ACTS[act], 0)
    awq._check(lib().awq_gemm_fused(x.data_ptr(), _ptr(inv_s_c), packed.data_ptr(), m, n, k, group, fmt, tail,
                                    y.data_ptr(), _ptr(ws), ws_bytes, awq._stream(index)), "awq_gemm_fused")
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
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k is required")
    if (k_cache is None) != (v_cache is None):
        raise ValueError("k_cache and v_cache go together")
    if k is None and (k_cache is not None or k_out is not None):
        raise ValueError("a cache or k_out needs k")
    if k_cache is not None and (v is None or slots is None):
        raise ValueError("a cache needs v and slots")
    dtype, index = ref.dtype, ref.get_device()
    if not (index >= 0 and dtype in DT and ref.dim() == 3 and (q is None or _packed(q, dtype, index))
            and (k is None or _packed(k, dtype, index)) and (v is None or _packed(v, dtype, index))):
        _refuse(ref, dtype, [(n, t) for n, t in (("q", q), ("k", k), ("v", v)) if t is not None])
    tokens, _, d = ref.shape
    if not (_vector(positions, torch.int32, index, (tokens,))
            and _vector(inv_freq, torch.float32, index, (len(inv_freq),))
            and (slots is None or _vector(slots, torch.int64, index, (tokens,)))):
        _refuse(ref, dtype, (), (("positions", positions, torch.int32, (tokens,)),
                                 ("inv_freq", inv_freq, torch.float32, (inv_freq.numel(),)),
                                 ("slots", slots, torch.int64, (tokens,))))
    rot_dim = 2 * len(inv_freq)
    if rot_dim > d:
        raise ValueError("inv_freq has more pairs than the head")
    q_heads = kv_heads = pages = page_size = q_ptr = qo_ptr = k_ptr = ko_ptr = v_ptr = kc_ptr = vc_ptr = 0
    qs = qos = ks = kos = vs = (0, 0)
    cache = (0, 0, 0)
    if q is not None:
        q_out = _output(q_out, "q_out", q, index)
        q_heads = q.shape[1]
        q_ptr, qo_ptr, qs, qos = q.data_ptr(), q_out.data_ptr(), _strides(q, q_heads, d), _strides(q_out, q_heads, d)
    if k is not None:
        kv_heads = k.shape[1]
        if k.shape[0] != tokens or k.shape[2] != d:
            raise ValueError("k must have q's tokens and head size")
        k_ptr, ks = k.data_ptr(), _strides(k, kv_heads, d)
        if k_cache is None or k_out is not None:
            k_out = _output(k_out, "k_out", k, index)
            ko_ptr, kos = k_out.data_ptr(), _strides(k_out, kv_heads, d)
        if k_cache is not None:
            awq._shape(v, "v", k.shape)
            pages, page_size, *cache = _cache(k_cache, v_cache, dtype, kv_heads, d, index)
            kc_ptr, vc_ptr, v_ptr, vs = k_cache.data_ptr(), v_cache.data_ptr(), v.data_ptr(), _strides(v, kv_heads, d)
    args = _ROPE.pack(q_ptr, qo_ptr, k_ptr, ko_ptr, v_ptr, kc_ptr, vc_ptr, positions.data_ptr(),
                      inv_freq.data_ptr(), _ptr(slots), tokens, *qs, *qos, *ks, *kos, *vs, *cache, pages,
                      page_size, q_heads, kv_heads, d, rot_dim, DT[dtype], interleaved, inverse, scale, 0)
    awq._check(lib().awq_rope(args, awq._stream(index)), "awq_rope")
    return q_out, k_out


def awq_attn_prompt(q, k, v, cu_seqlens, scale: float | None = None, out=None) -> torch.Tensor:
    """Causal attention of packed prompts: q [tokens, q_heads, D], k and v [tokens, kv_heads,
    D]; sequence b is the tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32 [seqs + 1]).
    scale defaults to D ** -0.5. Tokens in no sequence are not written."""
    dtype, index = q.dtype, q.get_device()
    if not (index >= 0 and dtype in DT and _packed(q, dtype, index) and _packed(k, dtype, index)
            and _packed(v, dtype, index)):
        _refuse(q, dtype, (("q", q), ("k", k), ("v", v)))
    tokens, hq, d = q.shape
    hkv = k.shape[1]
    if k.shape[0] != tokens or k.shape[2] != d or v.shape != k.shape:
        awq._shape(k, "k", (tokens, hkv, d))
        awq._shape(v, "v", (tokens, hkv, d))
    points = len(cu_seqlens)
    if points < 1:
        raise ValueError("cu_seqlens must be [seqs + 1]")
    if not _vector(cu_seqlens, torch.int32, index, (points,)):
        _refuse(q, dtype, (), (("cu_seqlens", cu_seqlens, torch.int32, (points,)),))
    out = _output(out, "out", q, index)
    args = _PROMPT.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), cu_seqlens.data_ptr(), tokens,
                        points - 1, *_strides(q, hq, d), *_strides(k, hkv, d), *_strides(v, hkv, d),
                        *_strides(out, hq, d), hq, hkv, d, DT[dtype], d ** -0.5 if scale is None else scale, 0)
    awq._check(lib().awq_attn_prompt(args, awq._stream(index)), "awq_attn_prompt")
    return out


@functools.lru_cache(maxsize=None)
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
    tokens see those up to themselves. A token that sees nothing gets zeros. ws: uint8,
    awq_attn_tree_workspace_bytes() of them (cached per device and stream when absent)."""
    dtype, index = q.dtype, q.get_device()
    if not (index >= 0 and dtype in DT and _packed(q, dtype, index)):
        _refuse(q, dtype, (("q", q),))
    tokens, hq, d = q.shape
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, D]")
    hkv = k_cache.shape[1]
    pages, page_size, *cache = _cache(k_cache, v_cache, dtype, hkv, d, index)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [seqs, width]")
    seqs, width = block_table.shape
    i32 = torch.int32
    if not (_vector(block_table, i32, index, (seqs, width)) and _vector(ctx_lens, i32, index, (seqs,))
            and _vector(cu_q, i32, index, (seqs + 1,))
            and (mask is None or _vector(mask, torch.int64, index, (tokens,)))):
        _refuse(q, dtype, (), (("block_table", block_table, i32, (seqs, width)), ("ctx_lens", ctx_lens, i32, (seqs,)),
                               ("cu_q", cu_q, i32, (seqs + 1,)), ("mask", mask, torch.int64, (tokens,))))
    out = _output(out, "out", q, index)
    if ws is None:
        need = awq_attn_tree_workspace_bytes(tokens, seqs, width, page_size, max_q, hq, hkv, d)
        ws = _workspace(need, index) if need else None
    else:
        awq._dev(ws, "ws", torch.uint8)
        awq._same_device(q, ws=ws)
    ws_ptr, ws_bytes = (0, 0) if ws is None else (ws.data_ptr(), ws.numel())
    args = _TREE.pack(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), block_table.data_ptr(),
                      ctx_lens.data_ptr(), cu_q.data_ptr(), _ptr(mask), ws_ptr, ws_bytes, tokens, seqs, width, pages,
                      *_strides(q, hq, d), *_strides(out, hq, d), *cache, page_size, max_q, hq, hkv, d, DT[dtype],
                      d ** -0.5 if scale is None else scale, 0)
    awq._check(lib().awq_attn_tree(args, awq._stream(index)), "awq_attn_tree")
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


def _workspace(need: int, index: int) -> torch.Tensor:
    """A workspace of at least `need` bytes, cached per device and stream and grown on
    demand, as awq.workspace."""
    key = (index, awq._stream(index))
    cur = _WS.get(key)
    if cur is None or cur.numel() < need:
        cur = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=torch.device("cuda", index))
        _WS[key] = cur
    return cur
