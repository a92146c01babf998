"""Plain float64 forms of the feed-forward operators, with the error bounds that the kernels'
arithmetic gives (derived here, from the formats alone). E is float32's rounding, 2^-24."""
import torch

import block_ref
from block_ref import ACTS, TINY, U, check, cpu64  # noqa: F401

E = 2.0 ** -24


def norm(x, weight, eps, residual=None):
    """(h, v, bound of v in float32). h is the sum as an element (float32 holds it to one rounding,
    as torch's conversion does). The squares' sum is a chain of at most 32 additions per thread, 6
    across lanes and 16 across wavefronts: 54 E, half of it in the root; the root, the division
    and the two products add 6 E."""
    dtype = x.dtype
    h = cpu64(x)
    if residual is not None:
        h = (x.detach().cpu().float() + residual.detach().cpu().float()).to(dtype).double()
    v = h * (h.square().mean(1, keepdim=True) + eps).rsqrt()
    if weight is not None:
        v = v * cpu64(weight)
    return h.to(dtype), v, 34 * E * v.abs()


def check_rows8(q, scale, v, off, what=""):
    """8-bit rows of v, known to `off`: the scale is max|v| / 127 within its rounding, and a code is
    the nearest step to v within half a step and what v and the step may be off."""
    q, scale = q.detach().cpu().double(), scale.detach().cpu().double()
    want = v.abs().amax(1) / 127
    assert bool(((scale - want).abs() <= (off.amax(1) / 127) + 2 * E * want + 2.0 ** -149).all()), what
    slack = off + 2 * (127 * 4 * E) * want[:, None]
    assert bool(((q * want[:, None] - v).abs() <= 0.5 * want[:, None] + slack).all()), what
    assert bool((q.abs().amax(1)[want > 0] == 127).all()), what


def tail(v, dtype, act, bias, mul, residual, off):
    """(value, bound) of act(v + bias) * mul + residual for v within `off`; the activations' slopes
    are at most 1.13, the hardware's exponential and reciprocal add 2e-6 of the value."""
    y = v if bias is None else v + cpu64(bias)
    pre = y.abs()
    bound = 1.13 * (off + 2e-6 * pre)
    y = ACTS[act](y)
    if mul is not None:
        y, bound = y * cpu64(mul), bound * cpu64(mul).abs()
    if residual is not None:
        y = y + cpu64(residual)
    return y, bound + 4 * E * y.abs() + U[dtype] * y.abs() + TINY[dtype]


def gemm_i8(q, scale, w, s_w, dtype, act="none", bias=None, mul=None, residual=None):
    """w int8 [N, K], s_w [N]. The sum is exact; its conversion and the two scales round."""
    v = cpu64(q) @ cpu64(w).t() * cpu64(scale)[:, None] * cpu64(s_w)
    return tail(v, dtype, act, bias, mul, residual, 4 * E * v.abs())


def unpack_i8(packed, n, k):
    """(w int8 [n, k], scales [n]) of a packed layer, byte by byte from the header's description."""
    raw = packed.detach().cpu()
    units = -(-k // 64)
    rows, kk = torch.arange(n)[:, None], torch.arange(k)
    at = (rows // 16 * units + kk // 64) * 1024 + 16 * (16 * (kk % 64 // 16) + rows % 16) + kk % 16
    base = -(-n // 16) * units * 1024
    return raw.view(torch.int8)[at], raw[base:base + 4 * n].view(torch.float32)


def route(x, w, k, bias=None, score="softmax", renormalize=True, scale=1.0):
    logits = cpu64(x) @ cpu64(w).t()
    p = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)
    choice = p if score == "sigmoid" else logits
    if bias is not None:
        choice = choice + cpu64(bias)
    behind = torch.where(torch.isnan(choice), -torch.inf, choice)
    ids = torch.empty(x.shape[0], k, dtype=torch.int32)
    for t in range(x.shape[0]):   # largest first, NaN behind -infinity, then the lowest index
        order = sorted(range(w.shape[0]), key=lambda e: (bool(torch.isnan(choice[t, e])), -float(behind[t, e]), e))
        ids[t] = torch.tensor(order[:k])
    weights = torch.gather(p, 1, ids.long())
    if renormalize:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total == 0, 0.0, weights / total)
    return ids, weights * scale


def moe(x, ids, weights, gate, up, down, act="silu", inv_in=None, inv_down=None, residual=None):
    """(value, bound); gate, up [E, F, H] and down [E, H, F] are the dequantized binary16 weights.
    Sums of F or H products in float32 err by (products + 64) E of their absolute terms."""
    dtype, u = torch.float16, U[torch.float16]
    tokens, hidden = x.shape
    y = torch.zeros(tokens, hidden, dtype=torch.float64)
    err = torch.zeros_like(y)
    big = torch.zeros_like(y)
    for t in range(tokens):
        for j in range(ids.shape[1]):
            e, wt = int(ids[t, j]), float(weights[t, j])
            if not 0 <= e < gate.shape[0]:
                continue
            xs = cpu64(x[t])
            if inv_in is not None:
                xs = (xs * cpu64(inv_in if inv_in.dim() == 1 else inv_in[e])).half().double()
            wg, wu, wd = cpu64(gate[e]), cpu64(up[e]), cpu64(down[e])
            g, v = wg @ xs, wu @ xs
            dg, dv = ((hidden + 64) * E * (m.abs() @ xs.abs()) for m in (wg, wu))
            a = ACTS[act](g)
            da = 1.13 * dg + 2e-6 * g.abs()
            m = a * v
            dm = da * v.abs() + (a.abs() + da) * dv
            if inv_down is not None:
                f = cpu64(inv_down if inv_down.dim() == 1 else inv_down[e])
                m, dm = m * f, dm * f.abs()
            # the operand of the second product is binary16: a value near a border may round the other way
            dm = dm + 4 * E * m.abs()
            r = m.half().double()
            dm = torch.where(dm > 0, dm + 2 * u * m.abs() + 2 * TINY[dtype], dm)
            y[t] += wt * (wd @ r)
            terms = wd.abs() @ r.abs()
            err[t] += abs(wt) * (wd.abs() @ dm + (down.shape[2] + 64) * E * terms)
            big[t] += abs(wt) * terms
    if residual is not None:
        y = y + cpu64(residual)
    return y, err + 64 * E * big + (u + 2 * E) * y.abs() + TINY[dtype]
