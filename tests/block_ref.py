"""Plain float64 forms of the decoder-block operators, with the error bounds that the
kernels' arithmetic gives (derived here, from the formats alone).

u is the rounding of the element type (2^-11 binary16, 2^-8 bfloat16). Float32 work inside
the kernels adds a few 2^-24 per operation; 2e-5 of the sums' absolute terms covers chains
of up to 128 products and the hardware's exponential and trigonometry (about 2^-21)."""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half the smallest subnormal


def cpu64(t):
    return t.detach().to("cpu", torch.float64)


def rope(x, positions, inv_freq, interleaved=False, inverse=False, scale=1.0):
    """(value, bound) of rotated x [tokens, heads, D]."""
    xf, rot = cpu64(x), 2 * inv_freq.numel()
    angle = positions.cpu().double()[:, None, None] * inv_freq.cpu().double()
    cos, sin = scale * torch.cos(angle), scale * torch.sin(-angle if inverse else angle)
    out = xf.clone()
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = xf[..., first], xf[..., second]
    out[..., first], out[..., second] = a * cos - b * sin, b * cos + a * sin
    bound = U[x.dtype] * out.abs() + TINY[x.dtype]
    both = 2e-6 * abs(scale) * (a.abs() + b.abs())
    bound[..., first] += both
    bound[..., second] += both
    bound[..., rot:] = 0.0
    return out, bound


def attend(q, k, v, sees, scale, dtype):
    """(value, bound) of one head: q [n, D], k and v [m, D], sees [n, m]. Keys and values that
    no row sees may hold anything. Probabilities are rounded to the element type before
    they meet v (in units of 2^-7 of the row's maximum: binary16's subnormals add 2^-32 of
    it, eight times that where the maximum in use lags by 2^8 ... the other way only), and
    scores carry float32 errors of |q| |k| scale 2^-18."""
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
    bound = torch.zeros_like(out)
    for i in range(q.shape[0]):
        at = sees[i].nonzero().flatten()
        if len(at) == 0:
            continue
        kk, vv = k[at], v[at]
        s = (kk @ q[i]) * scale
        p = torch.softmax(s, 0)
        out[i] = p @ vv
        slack = U[dtype] + 2e-5 + 2.0 ** -18 * float((kk.abs() @ q[i].abs()).max()) * scale
        least = 2.0 ** -32 * float(p.max()) * vv.abs().sum(0) if dtype == torch.float16 else 0.0
        bound[i] = slack * (p @ vv.abs()) + U[dtype] * out[i].abs() + least + TINY[dtype]
    return out, bound


def prompt(q, k, v, lengths, scale=None):
    q, k, v, dtype = cpu64(q), cpu64(k), cpu64(v), q.dtype
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    at = 0
    for n in lengths:
        sees = torch.ones(n, n, dtype=torch.bool).tril()
        for h in range(hq):
            g = h // (hq // hkv)
            o, b = attend(q[at:at + n, h], k[at:at + n, g], v[at:at + n, g], sees, scale, dtype)
            out[at:at + n, h], bound[at:at + n, h] = o, b
        at += n
    return out, bound


def tree(q, k_cache, v_cache, table, ctx, drafts, masks, scale=None):
    """masks: a python int of bits per token, or None for the chain."""
    dtype = q.dtype
    q, kc, vc, table = cpu64(q), cpu64(k_cache), cpu64(v_cache), table.cpu()
    hq, hkv, d, page = q.shape[1], kc.shape[1], q.shape[2], kc.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    at = 0
    for b, (c, t) in enumerate(zip(ctx, drafts)):
        n = c + t
        pages = table[b, :(n + page - 1) // page].long()
        sees = torch.zeros(t, n, dtype=torch.bool)
        sees[:, :c] = True
        for i in range(t):
            bits = (1 << (i + 1)) - 1 if masks is None else masks[at + i]
            for j in range(t):
                sees[i, c + j] = bool(bits >> j & 1)
        for h in range(hq):
            g = h // (hq // hkv)
            k, v = kc[pages, g].reshape(-1, d)[:n], vc[pages, g].reshape(-1, d)[:n]
            o, e = attend(q[at:at + t, h], k, v, sees, scale, dtype)
            out[at:at + t, h], bound[at:at + t, h] = o, e
        at += t
    return out, bound


ACTS = {
    "none": lambda t: t,
    "relu": torch.relu,
    "gelu": lambda t: 0.5 * t * torch.erfc(-t / math.sqrt(2.0)),
    "gelu_tanh": lambda t: 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))),
    "silu": lambda t: t * torch.sigmoid(t),
}


def tail(v, act, bias, mul, residual, off):
    """(value, bound) of act(v + bias) * mul + residual for sums that are within `off` of v.
    The activations' slopes are at most 1.13."""
    y = v if bias is None else v + cpu64(bias)
    pre = y.abs()
    y = ACTS[act](y)
    bound = 1.13 * (off + 2e-6 * pre)
    if mul is not None:
        y, bound = y * cpu64(mul), bound * cpu64(mul).abs()
    if residual is not None:
        y = y + cpu64(residual)
    return y, bound + U[torch.float16] * y.abs() + 2e-7 * pre + TINY[torch.float16]


def check(got, want, bound, what=""):
    """Elementwise |got - want| <= bound, with the same places finite."""
    g = cpu64(got)
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what
    bad = (g - want).abs() > bound
    bad &= ~torch.isnan(want)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} past the bound, first at {i}: "
                             f"{float(g[i])} against {float(want[i])} +- {float(bound[i])}")
