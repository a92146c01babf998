"""Norms, 8-bit rows and the product in 8-bit integers (``awq_ffn.h``).

Same manner as ``block``: each function has the name of its C entry point, checks device, dtype,
layout and extents, allocates outputs with PyTorch, runs on PyTorch's current stream and raises
``AwqError`` on a non-zero status. Elements are float16 or bfloat16; rows may be strided views
whose last dimension is contiguous.

    y, _, _, h = int8.awq_rms_norm(x, weight, residual=h)              # for a W4A16 layer
    _, q, s, h = int8.awq_rms_norm(x, weight, residual=h, y16=False, i8=True)
    y = int8.awq_gemm_i8(q, s, int8.awq_pack_i8(w), n, k, residual=h)  # for prompts
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import awq
from .block import ACTS, DT, _block

EXPORTS = ("awq_gemm_i8", "awq_gemm_i8_workspace_bytes", "awq_pack_i8", "awq_packed_i8_bytes", "awq_quant_i8",
           "awq_rms_norm")


class Rows(NamedTuple):
    """What awq_rms_norm returns; None where it was not asked for."""
    y: torch.Tensor | None       # the norm in the input's type
    q: torch.Tensor | None       # the norm in 8 bits, int8
    scale: torch.Tensor | None   # float32 [tokens]
    h: torch.Tensor | None       # x + residual


def awq_rms_norm(x, weight=None, eps: float = 1e-5, residual=None, *, y16: bool = True, i8: bool = False, y=None,
                 q=None, scale=None, h=None) -> Rows:
    """Root-mean-square norm of the rows of x [tokens, width]: with h = x + residual (rounded to
    the type; x without a residual), v = h * weight / sqrt(mean(h^2) + eps). y16 asks for v in
    the type (y), i8 for int8 codes q = rint(v / scale), scale = max|v| / 127 of each row. h may
    be x or residual itself, and so may y. A factor for each channel in front of the next product
    (inv_s_c of a folded weight) goes into `weight`."""
    return Rows(*_block.rms_norm(x, weight, eps, residual, y16, i8, y, q, scale, h))


def awq_quant_i8(x, inv_s_c=None, *, q=None, scale=None):
    """(q int8 [tokens, width], scale float32 [tokens]) of the rows of x * inv_s_c (of x's type,
    [width])."""
    return _block.quant_i8(x, inv_s_c, q, scale)


@functools.lru_cache(maxsize=4096)
def awq_packed_i8_bytes(n: int, k: int) -> int:
    fn = awq.lib().awq_packed_i8_bytes
    fn.restype, fn.argtypes = ctypes.c_size_t, [ctypes.c_int64] * 2
    return int(fn(n, k))


def awq_pack_i8(w, s_c=None) -> torch.Tensor:
    """w [N, K] (times s_c [K]) in 8 bits with a scale for each output, as awq_gemm_i8 reads it
    (uint8)."""
    return _block.pack_i8(w, s_c)


@functools.lru_cache(maxsize=4096)
def awq_gemm_i8_workspace_bytes(m: int, n: int, k: int) -> int:
    fn = awq.lib().awq_gemm_i8_workspace_bytes
    fn.restype, fn.argtypes = ctypes.c_size_t, [ctypes.c_int64] * 3
    return int(fn(m, n, k))


def awq_gemm_i8(q, scale, packed, n: int, k: int, *, bias=None, act: str = "none", mul=None, residual=None,
                dtype: torch.dtype = torch.float16, y=None, ws=None) -> torch.Tensor:
    """y [M, N] = act(scale * s_w * (q . w^T) + bias) * mul + residual, rounded once to `dtype`,
    the type of bias [N], mul and residual [M, N]. y may be mul or residual itself. ws: uint8,
    awq_gemm_i8_workspace_bytes() of them; when absent, awq.scratch."""
    code, kind = ACTS.get(act), DT.get(dtype)
    if code is None:
        raise ValueError(f"act must be one of {tuple(ACTS)}")
    if kind is None:
        raise TypeError("dtype must be torch.float16 or torch.bfloat16")
    return _block.gemm_i8(q, scale, packed, n, k, bias, code, mul, residual, kind, y, ws)


class Int8Linear:
    """A linear layer in 8 bits: rows are quantized as they come (or come quantized, from
    awq_rms_norm), y = x . w^T. It keeps a byte for each weight; beside an awq.QuantLinear of the same
    weights, which single tokens take, that is about three times the 4-bit layer's bytes in all."""

    def __init__(self, packed, n: int, k: int, inv_s_c=None):
        self.packed, self.n, self.k, self.inv_s_c = packed, n, k, inv_s_c

    @classmethod
    def from_weight(cls, w, s_c=None, inv_s_c=None):
        """s_c and inv_s_c of w's type (awq.awq_channel_scale forms them in float16): folded into
        the weight, and applied to rows that this layer quantizes itself."""
        return cls(awq_pack_i8(w, s_c), w.shape[0], w.shape[1], inv_s_c)

    def __call__(self, x, scale=None, *, bias=None, act="none", mul=None, residual=None, dtype=None, y=None):
        """x [M, K] in float16 or bfloat16, or int8 with its `scale` [M] (then `dtype` is the
        output's, float16 unless given)."""
        if scale is None:
            dtype = x.dtype if dtype is None else dtype
            x, scale = awq_quant_i8(x, self.inv_s_c)
        return awq_gemm_i8(x, scale, self.packed, self.n, self.k, bias=bias, act=act, mul=mul, residual=residual,
                           dtype=torch.float16 if dtype is None else dtype, y=y)
