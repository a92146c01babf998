"""Mixture of experts: the router, and the layer of W4A16 experts for a few tokens
(``awq_ffn.h``). Same manner as ``block`` and ``int8``.

    ids, weights = moe.awq_moe_route(x, router, k=2)
    y = moe.awq_moe(x, ids, weights, gate, up, down, ffn, residual=h)
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import awq
from .block import ACTS, _block

EXPORTS = ("awq_moe", "awq_moe_route", "awq_moe_route_workspace_bytes", "awq_moe_workspace_bytes")
SCORES = {"softmax": 0, "sigmoid": 1}
MAX_TOKENS = 64
MAX_K = 32


@functools.lru_cache(maxsize=4096)
def awq_moe_route_workspace_bytes(tokens: int, hidden: int, experts: int) -> int:
    fn = awq.lib().awq_moe_route_workspace_bytes
    fn.restype, fn.argtypes = ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
    return int(fn(tokens, hidden, experts))


def awq_moe_route(x, w, k: int, bias=None, *, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                  ids=None, weights=None, ws=None):
    """(ids int32 [tokens, k], weights float32 [tokens, k]): the k experts of each token with the
    largest logits x . w^T (x [tokens, hidden], w [experts, hidden]; score "softmax"), or with the
    largest sigmoids of them (score "sigmoid"), in that order, ties to the lowest index. bias
    (float32 [experts]) is added to the logits or sigmoids for the choice alone. weights are
    scale times the chosen scores, divided by their sum if `renormalize`. Logits are summed in float64."""
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {tuple(SCORES)}")
    return _block.moe_route(x, w, k, bias, code, renormalize, scale, ids, weights, ws)


@functools.lru_cache(maxsize=4096)
def awq_moe_workspace_bytes(tokens: int, hidden: int, ffn: int, k: int) -> int:
    fn = awq.lib().awq_moe_workspace_bytes
    fn.restype, fn.argtypes = ctypes.c_size_t, [ctypes.c_int64] + [ctypes.c_int32] * 3
    return int(fn(tokens, hidden, ffn, k))


def awq_moe(x, ids, weights, gate, up, down, ffn: int, group: int = awq.GROUP, fmt: int = awq.FMT_ASYM, *,
            act: str = "silu", inv_in=None, inv_down=None, residual=None, y=None, ws=None) -> torch.Tensor:
    """y[t] = residual[t] + sum over j of weights[t][j] * down[e](act(gate[e](x[t])) * up[e](x[t]))
    with e = ids[t][j], for up to 64 tokens x fp16 [tokens, hidden]. gate and up: uint8 [experts,
    awq.awq_repacked_bytes(ffn, hidden, group, fmt)], down: uint8 [experts,
    awq.awq_repacked_bytes(hidden, ffn, group, fmt)] of packed layers. inv_in ([experts, hidden] or
    [hidden]) and inv_down ([experts, ffn] or [ffn]) are the layers' inverse channel scales. An id
    outside the experts takes part in nothing; a token may name an expert twice. y may be x or
    residual itself."""
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {tuple(ACTS)}")
    return _block.moe_layer(x, ids, weights, gate, up, down, ffn, group, fmt, code, inv_in, inv_down, residual, y, ws)


class MoeLayer:
    """Experts with their router: y = residual + sum of the k best experts' outputs."""

    def __init__(self, router, gate, up, down, ffn, k, group=awq.GROUP, fmt=awq.FMT_ASYM, *, bias=None,
                 score="softmax", renormalize=True, scale=1.0, act="silu", inv_in=None, inv_down=None):
        """bias, score, renormalize and scale are awq_moe_route's, the others awq_moe's."""
        self.router, self.gate, self.up, self.down = router, gate, up, down
        self.ffn, self.k, self.group, self.fmt = ffn, k, group, fmt
        self.bias, self.score, self.renormalize, self.scale = bias, score, renormalize, scale
        self.act, self.inv_in, self.inv_down = act, inv_in, inv_down

    @classmethod
    def from_weights(cls, router, gate, up, down, k, group=awq.GROUP, fmt=awq.FMT_ASYM, *, s_in=None, s_down=None, **kw):
        """router fp16 [experts, hidden]; gate and up fp16 [experts, ffn, hidden], down fp16
        [experts, hidden, ffn], quantized and packed here. s_in ([experts, hidden] or [hidden]) and
        s_down ([experts, ffn] or [ffn]) are channel scales folded into gate and up, and into down;
        their inverses (awq.awq_channel_scale forms both) go with them as inv_in and inv_down.
        inv_in or inv_down without its scale belongs to weights that carry the scale already."""
        def stack(w, s):
            n, kk = w.shape[1:]
            scales = [None if s is None else s if s.dim() == 1 else s[e] for e in range(w.shape[0])]
            return torch.stack([awq.awq_repack(*awq.awq_pack(e, s_c, group, fmt), n, kk, group, fmt)
                                for e, s_c in zip(w, scales)])
        return cls(router, stack(gate, s_in), stack(up, s_in), stack(down, s_down), gate.shape[1], k, group, fmt, **kw)

    def __call__(self, x, residual=None):
        """x fp16 [tokens, hidden]; more tokens than one call takes go in several."""
        ids, weights = awq_moe_route(x, self.router, self.k, self.bias, score=self.score,
                                     renormalize=self.renormalize, scale=self.scale)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        for at in range(0, x.shape[0], MAX_TOKENS):
            part = slice(at, at + MAX_TOKENS)
            awq_moe(x[part], ids[part], weights[part], self.gate, self.up, self.down, self.ffn, self.group, self.fmt,
                    act=self.act, inv_in=self.inv_in, inv_down=self.inv_down,
                    residual=None if residual is None else residual[part], y=y[part])
        return y
