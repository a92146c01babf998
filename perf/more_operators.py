"""Workloads of the operators of a decoder's feed-forward half: root-mean-square norm with the
residual's addition and an output in 8 bits, the product in 8-bit integers, the router of a
mixture of experts, and the experts' layer for a few tokens.

Each case is one call of one operator. `run` computes it in its plain form (elementary torch
operations, sums in float32, rounded once at the end), or, where `own` is true, with the
package's kernels. `exact` computes the same outputs from the definitions in float64.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


def listed():
    return [
        # the norm before a projection of one token of a 7B block (latency)
        dict(name="rows_token_f16", op="rows", tokens=1, width=4096, norm=True, residual=True, i8=False, dtype="f16"),
        # the norm of a long prompt of a 70B block
        dict(name="rows_long_bf16", op="rows", tokens=16384, width=8192, norm=True, residual=True, i8=False,
             dtype="bf16"),
        # the norm before the 8-bit product of a ragged batch of prompts
        dict(name="rows_norm_i8_bf16", op="rows", tokens=1557, width=4096, norm=True, residual=True, i8=True,
             dtype="bf16"),
        # a gated activation on its way into the 8-bit down projection
        dict(name="rows_quant_f16", op="rows", tokens=2048, width=14336, norm=False, residual=False, i8=True,
             dtype="f16"),
        # output projection of one token in 8 bits, with its residual (latency)
        dict(name="i8_token_f16", op="i8", m=1, n=4096, k=4096, act="none", bias=False, mul=False, residual=True,
             dtype="f16"),
        # down projection of a ragged batch of short prompts
        dict(name="i8_ragged_bf16", op="i8", m=333, n=4096, k=11008, act="none", bias=False, mul=False,
             residual=True, dtype="bf16"),
        # gate projection of a prompt: silu(gate) * up
        dict(name="i8_gate_m2048_f16", op="i8", m=2048, n=14336, k=4096, act="silu", bias=False, mul=True,
             residual=False, dtype="f16"),
        # one token's choice among a few large experts (latency)
        dict(name="route_token_f16", op="route", tokens=1, hidden=4096, experts=8, k=2, sigmoid=False, dtype="f16"),
        # a batch of prompts over many small experts, scores by sigmoid with a balancing bias
        dict(name="route_prompt_bf16", op="route", tokens=517, hidden=4096, experts=128, k=8, sigmoid=True,
             dtype="bf16"),
        # one token through two of eight large experts
        dict(name="moe_token", op="moe", tokens=1, hidden=4096, ffn=14336, experts=8, k=2, shards=1, group=128,
             sym=False, residual=True),
        # a few sequences over small experts, half of which another device holds
        dict(name="moe_few", op="moe", tokens=7, hidden=2048, ffn=1408, experts=32, k=6, shards=2, group=64,
             sym=True, residual=False),
        # batched decode: nearly every expert has tokens
        dict(name="moe_batch", op="moe", tokens=48, hidden=4096, ffn=1536, experts=64, k=8, shards=1, group=128,
             sym=False, residual=True),
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm; long sizes are ragged (no multiples of 1024)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v - 1 if v % 1024 == 0 and v > lo else v


def draw(rng):
    op = rng.choice(["rows", "i8", "route", "moe"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rows":
        width = rng.choice([8 * _log(rng, 8, 2048), rng.choice([2048, 4096, 5120, 8192])])
        tokens = _log(rng, 1, min(16384, 16384 * 8192 // width))
        norm = rng.random() < 0.7
        i8 = not norm or (rng.random() < 0.5 and tokens * width <= 2048 * 14336)
        if i8:
            tokens = min(tokens, 2048 * 14336 // width)
        return dict(op=op, tokens=tokens, width=width, norm=norm, residual=norm and rng.random() < 0.7, i8=i8,
                    dtype=dtype)
    if op == "i8":
        n = 8 * _log(rng, 32, 14336 // 8)
        k = 16 * _log(rng, 16, 14336 // 16)
        m = _log(rng, 1, min(8192, 2048 * 14336 * 4096 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5, mul=rng.random() < 0.4,
                    residual=rng.random() < 0.5, dtype=dtype)
    experts = rng.choice([4, 8, 16, 32, 60, 64, 128])
    k = min(experts, rng.choice([1, 2, 2, 4, 6, 8]))
    if op == "route":
        hidden = rng.choice([8 * _log(rng, 32, 1024), 2048, 4096, 5120])
        return dict(op=op, tokens=_log(rng, 1, 2048), hidden=hidden, experts=experts, k=k,
                    sigmoid=rng.random() < 0.5, dtype=dtype)
    hidden = 128 * _log(rng, 2, 32)
    ffn = 128 * _log(rng, 1, max(2, min(112, 64 * 4096 * 1536 // (128 * experts * hidden))))
    return dict(op=op, tokens=_log(rng, 1, 64), hidden=hidden, ffn=ffn, experts=experts, k=k,
                shards=rng.choice([1, 1, 2]), group=rng.choice([32, 64, 128, 128]), sym=rng.random() < 0.3,
                residual=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "rows":
        elements = float(case["tokens"]) * case["width"]
        per = 2 + 4 * case["residual"] + (1 if case["i8"] else 2)
        return {"bytes": elements * per + 4 * case["tokens"] * case["i8"] + 2 * case["width"],
                "flops": elements * (4 + 2 * case["i8"])}
    if op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 1.0 * m * k + n * k + 4 * (m + n) + 2.0 * m * n * (1 + case["mul"] + case["residual"])
                + 2 * n * case["bias"], "flops": 2.0 * m * n * k}
    t, h, e, k = case["tokens"], case["hidden"], case["experts"], case["k"]
    if op == "route":
        return {"bytes": 2.0 * h * (t + e) + 8 * t * k + 4 * e * case["sigmoid"], "flops": 2.0 * t * e * h}
    # the experts that have tokens, as many as are expected
    share = k / (e * case["shards"])
    active = e * (1 - (1 - share) ** t)
    weight = 0.5 + (2.0 if case["sym"] else 2.5) / case["group"]
    return {"bytes": 3 * active * h * case["ffn"] * weight + 2.0 * t * h * (2 + case["residual"]) + 8 * t * k,
            "flops": 6.0 * t * k / case["shards"] * h * case["ffn"]}


# --------------------------------------------------------------------------- inputs

def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device=DEV)


def _stream(gen, tokens, width, dtype):
    """A residual stream: ~N(0, 1), a few channels much larger, tokens of different size."""
    gain = torch.ones(width, device=DEV)
    gain[torch.randperm(width, generator=gen, device=DEV)[:max(1, width // 200)]] = 20.0
    size = torch.exp(0.5 * torch.randn(tokens, 1, generator=gen, device=DEV))
    return _randn(gen, tokens, width).mul_(gain).mul_(size).to(dtype)


def _prepare_rows(case, gen):
    t, w, dt = case["tokens"], case["width"], DTYPES[case["dtype"]]
    s = dict(case=case, x=_stream(gen, t, w, dt), weight=None, residual=None, inv_s_c=None)
    if case["norm"]:
        s["weight"] = (1.0 + 0.2 * _randn(gen, w)).to(dt)
    else:
        s["inv_s_c"] = (0.25 + _rand(gen, w)).to(dt)
    if case["residual"]:
        s["residual"] = _stream(gen, t, w, dt)
    return s


def _prepare_i8(case, gen):
    m, n, k, dt = case["m"], case["n"], case["k"], DTYPES[case["dtype"]]
    q = (32.0 * _randn(gen, m, k)).round_().clamp_(-127, 127).to(torch.int8)
    # the packed layout of awq_pack_i8: 16 rows x 64 channels in 1024 bytes, lane l the 16 bytes
    # of row l % 16 from channel 16 (l / 16), rows and channels padded with zeros; then the scales
    rows, cols = -(-n // 16) * 16, -(-k // 64) * 64
    w = torch.zeros(rows, cols, dtype=torch.int8, device=DEV)
    w[:n, :k] = (40.0 * _randn(gen, n, k)).round_().clamp_(-127, 127).to(torch.int8)
    scales = torch.zeros(rows, device=DEV)
    scales[:n] = (0.5 + _rand(gen, n)) * (1.0 / (40.0 * math.sqrt(k)))
    codes = w.view(rows // 16, 16, cols // 64, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1)
    packed = torch.cat([codes.view(torch.uint8), scales.view(torch.uint8)])
    packed = torch.nn.functional.pad(packed, (0, -packed.numel() % 256))
    s = dict(case=case, q=q, scale=(0.5 + _rand(gen, m)) / 32.0, packed=packed, bias=None, mul=None, residual=None)
    if case["bias"]:
        s["bias"] = _randn(gen, n, dtype=dt)
    if case["mul"]:
        s["mul"] = _randn(gen, m, n, dtype=dt)
    if case["residual"]:
        s["residual"] = _randn(gen, m, n, dtype=dt)
    return s


def _prepare_route(case, gen):
    t, h, e, dt = case["tokens"], case["hidden"], case["experts"], DTYPES[case["dtype"]]
    return dict(case=case, x=_randn(gen, t, h, dtype=dt), w=(_randn(gen, e, h) * (1.5 / math.sqrt(h))).to(dt),
                bias=0.05 * _randn(gen, e) if case["sigmoid"] else None)


def _packed4(gen, experts, n, k, group, sym, gain):
    """[experts, bytes] of the packed layout of awq_repack: codes, scales and zeros, each region
    aligned to 256 bytes; codes around their zero points."""
    sets, tiles, units = max(1, 128 // group), (n + 15) // 16, k // 128
    size = tiles * units * 1024
    spread = [torch.randint(0, 6, (2, experts, size), generator=gen, device=DEV, dtype=torch.uint8) for _ in range(3)]
    nibbles = spread[0] + spread[1] + spread[2]
    parts = [nibbles[0] | (nibbles[1] << 4)]
    del spread, nibbles
    scales = gain * (0.5 + _rand(gen, experts, tiles * units * sets * 16)) / (3.0 * math.sqrt(k))
    parts.append(scales.to(torch.float16).view(torch.uint8))
    if not sym:
        zeros = torch.randint(6, 11, (2, experts, tiles * units * sets * 8), generator=gen, device=DEV,
                              dtype=torch.uint8)
        parts.append(zeros[0] | (zeros[1] << 4))
    return torch.cat([torch.nn.functional.pad(p, (0, -p.shape[1] % 256)) for p in parts], 1)


def _prepare_moe(case, gen):
    t, h, f, e, k = case["tokens"], case["hidden"], case["ffn"], case["experts"], case["k"]
    group, sym = case["group"], case["sym"]
    # a router's choice: some experts more in demand than others, and those past e held elsewhere
    scores = _randn(gen, t, e * case["shards"]) + 0.5 * _randn(gen, e * case["shards"])
    top, ids = torch.topk(scores, k, dim=1)
    return dict(case=case, x=_randn(gen, t, h, dtype=torch.float16),
                ids=torch.where(ids < e, ids, torch.full_like(ids, -1)).to(torch.int32),
                weights=torch.softmax(top, 1),
                gate=_packed4(gen, e, f, h, group, sym, 1.0), up=_packed4(gen, e, f, h, group, sym, 1.0),
                down=_packed4(gen, e, h, f, group, sym, 2.0),
                inv_down=(0.5 + _rand(gen, e, f)).to(torch.float16),
                residual=_randn(gen, t, h, dtype=torch.float16) if case["residual"] else None)


_PREPARE = {"rows": _prepare_rows, "i8": _prepare_i8, "route": _prepare_route, "moe": _prepare_moe}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return _PREPARE[case["op"]](case, gen)


# ----------------------------------------------------------------------- plain forms

def _values(q, scale, dtype):
    """What 8-bit codes and a scale for each row stand for."""
    return (q * scale[:, None]).to(dtype)


def _plain_rows(s):
    c, x, out = s["case"], s["x"], {}
    h = x
    if s["residual"] is not None:
        h = (x.float() + s["residual"].float()).to(x.dtype)
        out["h"] = h
    v = h.float()
    if c["norm"]:
        v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    else:
        v = v * s["inv_s_c"].float()
    if not c["i8"]:
        out["y"] = v.to(x.dtype)
        return out
    scale = v.abs().amax(1) / 127.0
    q = torch.round(v / scale.clamp_min(1e-30)[:, None]).to(torch.int8)
    return {**out, "values": _values(q, scale, x.dtype), "scale": scale}


def _act(v, name):
    if name == "relu":
        return v.clamp_min(0.0)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _plain_i8(s):
    c = s["case"]
    m, n, k = c["m"], c["n"], c["k"]
    tiles, units = -(-n // 16), -(-k // 64)
    w = s["packed"][:tiles * units * 1024].view(torch.int8).view(tiles, units, 4, 16, 16)
    w = w.permute(0, 3, 1, 2, 4).reshape(tiles * 16, units * 64)[:n, :k].float()
    scales = s["packed"][tiles * units * 1024:][:tiles * 64].view(torch.float32)[:n]
    y = (s["q"].float() @ w.t()) * s["scale"][:, None] * scales
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, c["act"])
    if s["mul"] is not None:
        y = y * s["mul"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["dtype"]])


def _plain_route(s):
    c = s["case"]
    # which expert is a border: 64 bits
    logits = s["x"].double() @ s["w"].double().t()
    if c["sigmoid"]:
        scores = 1.0 / (1.0 + torch.exp(-logits))
        choice = scores + s["bias"].double()
    else:
        top = logits.amax(1, keepdim=True)
        scores = torch.exp(logits - top)
        scores = scores / scores.sum(1, keepdim=True)
        choice = logits
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    weights = torch.gather(scores, 1, ids)
    return {"ids": ids.to(torch.int32), "weights": (weights / weights.sum(1, keepdim=True)).float()}


def _unpack4(packed, n, k, group, sym):
    """W_d [experts, n, k] as float32 of stacked packed layers: the binary16 values
    binary16((q - z) * s) that the format defines."""
    e, sets, tiles, units = packed.shape[0], max(1, 128 // group), (n + 15) // 16, k // 128
    size = tiles * units * 1024
    words = packed[:, :size].reshape(-1).view(torch.int32).view(e, tiles, units, 4, 16, 4)  # .., lane / 16, row, word
    # channel c of a word sits at nibble (c >> 1) + 4 (c & 1)
    shifts = torch.tensor([4 * ((c >> 1) + 4 * (c & 1)) for c in range(8)], dtype=torch.int32, device=DEV)
    q = ((words[..., None] >> shifts) & 15).half()
    which = torch.arange(4, device=DEV) * sets // 4                                         # the set of each quarter
    count = tiles * units * sets
    scales = packed[:, size:size + count * 32].reshape(-1).view(torch.float16).view(e, tiles, units, sets, 16)
    scales = scales[:, :, :, which]
    if sym:
        zeros = torch.full_like(scales, 8.0)
    else:
        at = size + (count * 32 + 255) // 256 * 256
        bits = packed[:, at:at + count * 8].reshape(e, tiles, units, sets, 8, 1)
        zeros = torch.cat([bits & 15, bits >> 4], -1).view(e, tiles, units, sets, 16).half()[:, :, :, which]
    w = ((q - zeros[..., None, None]) * scales[..., None, None]).float()                    # differences are exact
    return w.permute(0, 1, 4, 2, 3, 5, 6).reshape(e, tiles * 16, k)[:, :n]


def _plain_moe(s):
    c = s["case"]
    h, f, e, group, sym = c["hidden"], c["ffn"], c["experts"], c["group"], c["sym"]
    x = s["x"].float()
    g = x @ _unpack4(s["gate"], f, h, group, sym).transpose(1, 2)          # [experts, tokens, ffn]
    u = x @ _unpack4(s["up"], f, h, group, sym).transpose(1, 2)
    a = (_act(g, "silu") * u * s["inv_down"].float()[:, None]).half().float()   # binary16 by definition
    y = a @ _unpack4(s["down"], h, f, group, sym).transpose(1, 2)          # [experts, tokens, hidden]
    share = torch.zeros(c["tokens"], e + 1, device=DEV)                    # column e: experts held elsewhere
    ids = torch.where(s["ids"] < 0, torch.full_like(s["ids"], e), s["ids"]).long()
    share.scatter_add_(1, ids, s["weights"])
    out = (y * share[:, :e].t()[..., None]).sum(0)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.half()


_PLAIN = {"rows": _plain_rows, "i8": _plain_i8, "route": _plain_route, "moe": _plain_moe}


# ------------------------------------------------------------- the package's operators

def _own_rows(s):
    from bit_weight_only_w4a16_amd import int8
    c, x = s["case"], s["x"]
    if not c["norm"]:
        q, scale = int8.awq_quant_i8(x, s["inv_s_c"])
        return {"values": _values(q, scale, x.dtype), "scale": scale}
    r = int8.awq_rms_norm(x, s["weight"], EPS, residual=s["residual"], y16=not c["i8"], i8=c["i8"])
    out = {} if s["residual"] is None else {"h": r.h}
    if c["i8"]:
        return {**out, "values": _values(r.q, r.scale, x.dtype), "scale": r.scale}
    return {**out, "y": r.y}


def _own_i8(s):
    from bit_weight_only_w4a16_amd import int8
    c = s["case"]
    return int8.awq_gemm_i8(s["q"], s["scale"], s["packed"], c["n"], c["k"], bias=s["bias"], act=c["act"],
                            mul=s["mul"], residual=s["residual"], dtype=DTYPES[c["dtype"]])


def _own_route(s):
    from bit_weight_only_w4a16_amd import moe
    c = s["case"]
    ids, weights = moe.awq_moe_route(s["x"], s["w"], c["k"], bias=s["bias"],
                                     score="sigmoid" if c["sigmoid"] else "softmax")
    return {"ids": ids, "weights": weights}


def _own_moe(s):
    from bit_weight_only_w4a16_amd import moe
    c = s["case"]
    return moe.awq_moe(s["x"], s["ids"], s["weights"], s["gate"], s["up"], s["down"], c["ffn"], c["group"],
                       int(c["sym"]), act="silu", inv_down=s["inv_down"], residual=s["residual"])


_OWN = {"rows": _own_rows, "i8": _own_i8, "route": _own_route, "moe": _own_moe}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ float64 definitions

def _exact_rows(s):
    c, out = s["case"], {}
    v = s["x"].double()
    if s["residual"] is not None:
        # the sum is an element of its own: rounded to the type once
        v = v + s["residual"].double()
        out["h"] = v
        v = v.float().to(s["x"].dtype).double()
    if c["norm"]:
        v = v / torch.sqrt((v * v).sum(1, keepdim=True) / c["width"] + EPS) * s["weight"].double()
    else:
        v = v * s["inv_s_c"].double()
    if not c["i8"]:
        out["y"] = v
        return out
    step = v.abs().amax(1, keepdim=True) / 127
    return {**out, "values": torch.round(v / torch.where(step > 0, step, 1.0)) * step, "scale": step[:, 0]}


def _tail64(y, s, name):
    act = {"none": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
           "gelu": lambda t: t * 0.5 * torch.erfc(-t / math.sqrt(2.0)),
           "gelu_tanh": lambda t: t * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3))}
    if s["bias"] is not None:
        y = y + s["bias"].double()
    y = act[name](y)
    if s["mul"] is not None:
        y = y * s["mul"].double()
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_i8(s):
    c = s["case"]
    n, k = c["n"], c["k"]
    units = -(-k // 64)
    rows, kk = torch.arange(n, device=DEV)[:, None], torch.arange(k, device=DEV)
    at = (rows // 16 * units + kk // 64) * 1024 + (kk % 64 // 16 * 16 + rows % 16) * 16 + kk % 16
    w = s["packed"].view(torch.int8)[at].float()
    base = -(-n // 16) * units * 1024
    sw = s["packed"][base:base + 4 * n].view(torch.float32).double()
    y = torch.zeros(c["m"], n, dtype=torch.float64, device=DEV)
    for k0 in range(0, k, 1024):   # sums of 1024 products of at most 127 x 127 are whole numbers below 2^24
        y += torch.mm(s["q"][:, k0:k0 + 1024].float(), w[:, k0:k0 + 1024].t().contiguous())
    return _tail64(y * s["scale"].double()[:, None] * sw, s, c["act"])


def _exact_route(s):
    c = s["case"]
    logits = torch.stack([(s["x"].double() * row).sum(1) for row in s["w"].double()], 1)
    scores = torch.sigmoid(logits) if c["sigmoid"] else torch.softmax(logits, 1)
    choice = (scores + s["bias"].double()) if c["sigmoid"] else logits
    ids, left = [], choice.clone()
    for _ in range(c["k"]):
        best = left.max(1, keepdim=True).values
        first = torch.where(left == best, torch.arange(left.shape[1], device=DEV), left.shape[1]).amin(1)
        ids.append(first)
        left[torch.arange(len(first), device=DEV), first] = -math.inf
    ids = torch.stack(ids, 1)
    w = scores[torch.arange(c["tokens"], device=DEV)[:, None], ids]
    return {"ids": ids.to(torch.int32), "weights": w / w.sum(1, keepdim=True)}


def _exact_layer4(buf, n, k, group, sym):
    """W_d [n, k] in float64 of one packed layer, element by element."""
    sets, units, tiles = max(1, 128 // group), k // 128, (n + 15) // 16
    scale_at = tiles * units * 1024
    zero_at = scale_at + (tiles * units * sets * 32 + 255) // 256 * 256
    rows, kk = torch.arange(n, device=DEV)[:, None], torch.arange(k, device=DEV)
    quarter, word, c = kk % 128 // 32, kk % 32 // 8, kk % 8
    nibble = c // 2 + 4 * (c % 2)
    unit = rows // 16 * units + kk // 128
    code = (buf[unit * 1024 + (16 * quarter + rows % 16) * 16 + 4 * word + nibble // 2] >> (4 * (nibble % 2))) & 15
    set_at = unit * sets + quarter * sets // 4
    scale = buf[scale_at:scale_at + tiles * units * sets * 32].view(torch.float16)[set_at * 16 + rows % 16].double()
    zero = 8.0
    if not sym:
        zero = ((buf[zero_at + set_at * 8 + rows % 16 // 2] >> (4 * (rows % 2))) & 15).double()
    return ((code.double() - zero) * scale).half().double()


def _exact_moe(s):
    c = s["case"]
    h, f, group, sym = c["hidden"], c["ffn"], c["group"], c["sym"]
    y = torch.zeros(c["tokens"], h, dtype=torch.float64, device=DEV)
    if s["residual"] is not None:
        y += s["residual"].double()
    for e in range(c["experts"]):
        token, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not token.numel():
            continue
        x = s["x"][token].double()
        g = torch.mm(x, _exact_layer4(s["gate"][e], f, h, group, sym).t().contiguous())
        u = torch.mm(x, _exact_layer4(s["up"][e], f, h, group, sym).t().contiguous())
        a = (g * torch.sigmoid(g) * u * s["inv_down"][e].double()).half().double()
        d = torch.mm(a, _exact_layer4(s["down"][e], h, f, group, sym).t().contiguous())
        y.index_add_(0, token, d * s["weights"][token, j].double()[:, None])
    return y


_EXACT = {"rows": _exact_rows, "i8": _exact_i8, "route": _exact_route, "moe": _exact_moe}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
