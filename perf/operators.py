"""Workloads of the decoder-block operators: quantized product with an epilogue, rotary
positions with the cache write, prompt attention, and attention of drafted tokens over a
paged cache.

Each case is one call of one operator. `run` computes it in its plain form (elementary
torch operations in float32, rounded once at the end), or, where `own` is true, with the
package's kernels. `exact` computes the same outputs from the definitions in float64.

Shared conventions: tokens are packed ([tokens, heads, head_dim]); the cache is
[pages, kv_heads, page, head_dim]; sequence lengths are texts ("5,17") so that a case
holds plain values only.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one token of a 7B block: rotate 32 + 32 heads and store k, v (latency)
        dict(name="rope_token_f16", op="rope", lengths="1", start=4099, q_heads=32, kv_heads=32,
             head_dim=128, rot_dim=128, interleaved=False, page=16, dtype="f16"),
        # a packed prompt batch, grouped heads, part of the head, interleaved pairs
        dict(name="rope_prompt_bf16", op="rope", lengths="1500,1,517,29", start=0, q_heads=32, kv_heads=8,
             head_dim=128, rot_dim=64, interleaved=True, page=16, dtype="bf16"),
        # a long prompt of a 70B block (64 query heads, 8 key heads) far into the context
        dict(name="rope_long_f16", op="rope", lengths="16384", start=65536, q_heads=64, kv_heads=8,
             head_dim=128, rot_dim=128, interleaved=False, page=64, dtype="f16"),
        # short chat turns packed together, one of a single token (latency)
        dict(name="prompt_short_f16", op="prompt", lengths="1,33,120,64,7", q_heads=32, kv_heads=32,
             head_dim=128, dtype="f16"),
        # ragged batch of prompts, grouped heads
        dict(name="prompt_ragged_bf16", op="prompt", lengths="2048,517,1,1331,64,1999", q_heads=32,
             kv_heads=8, head_dim=128, dtype="bf16"),
        # one long document
        dict(name="prompt_long_f16", op="prompt", lengths="8192", q_heads=32, kv_heads=8, head_dim=128,
             dtype="f16"),
        # plain decode of one sequence: one new token over a short cache (latency)
        dict(name="tree_token_f16", op="tree", contexts="517", drafts="1", q_heads=32, kv_heads=32,
             head_dim=128, page=16, dtype="f16"),
        # speculative decoding: trees of drafted tokens over ragged caches
        dict(name="tree_draft_bf16", op="tree", contexts="4096,1333,0,2051,3000,77,1024,2500",
             drafts="16,25,7,16,1,32,16,9", q_heads=32, kv_heads=8, head_dim=128, page=16, dtype="bf16"),
        # batched decode over long caches (the memory-bound end)
        dict(name="tree_long_f16", op="tree",
             contexts="32768,16384,30011,8192,20000,32001,4099,25000,32768,12345,16000,32767,28000,31,9000,24576",
             drafts="1,1,1,1,1,1,1,1,1,1,1,1,1,1,1,1", q_heads=64, kv_heads=8, head_dim=128, page=64,
             dtype="f16"),
        # output projection of one token with its residual
        dict(name="linear_o_m1", op="linear", m=1, n=4096, k=4096, group=128, sym=False, act="none",
             bias=False, mul=False, residual=True),
        # gate projection of a batch of tokens: silu(gate) * up
        dict(name="linear_gate_m16", op="linear", m=16, n=11008, k=4096, group=128, sym=False, act="silu",
             bias=False, mul=True, residual=False),
        # prefill projection with bias, activation and residual
        dict(name="linear_prefill_m2048", op="linear", m=2048, n=14336, k=4096, group=128, sym=False,
             act="gelu_tanh", bias=True, mul=False, residual=True),
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm; long sizes are ragged (no multiples of 1024)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v - 1 if v % 1024 == 0 and v > lo else v


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8, 16])
    return kv * rng.choice([1, 2, 3, 4, 8]), kv


def draw(rng):
    op = rng.choice(["rope", "prompt", "tree", "linear"])
    dtype = rng.choice(["f16", "bf16"])
    hq, hkv = _heads(rng)
    head_dim = rng.choice([64, 128, 128, 80, 96])
    page = rng.choice([8, 16, 32, 64])
    if op == "rope":
        total = _log(rng, 1, 16384 * 72 // (hq + 2 * hkv))
        parts = [max(1, min(total, _log(rng, 1, total))) for _ in range(rng.randint(0, 3))]
        lengths = [p for p in parts if p < total // 4] + [max(1, total // 2 + 1)]
        rot = rng.choice([head_dim, head_dim // 2, head_dim // 4])
        return dict(op="rope", lengths=",".join(map(str, lengths)), start=_log(rng, 1, 131072) - 1, q_heads=hq,
                    kv_heads=hkv, head_dim=head_dim, rot_dim=rot, interleaved=rng.random() < 0.5,
                    page=page, dtype=dtype)
    if op == "prompt":
        seqs = rng.choice([1, 2, 4, 7])
        top = _log(rng, 2, int(math.sqrt(32 * 8192 * 8192 / (hq * seqs)) * 0.9))
        top = min(top, 8192)
        lengths = [_log(rng, 1, top) for _ in range(seqs - 1)] + [top]
        return dict(op="prompt", lengths=",".join(map(str, lengths)), q_heads=hq, kv_heads=hkv,
                    head_dim=head_dim, dtype=dtype)
    if op == "tree":
        seqs = _log(rng, 1, 16)
        top = _log(rng, 1, max(64, 16 * 32768 * 8 // (seqs * hkv * 4)))
        top = min(top, 32768)
        ctx = [min(top, _log(rng, 1, top + 1) - 1) for _ in range(seqs)]
        most = rng.choice([1, 1, 8, 64])
        drafts = [_log(rng, 1, most) for _ in range(seqs)]
        return dict(op="tree", contexts=",".join(map(str, ctx)), drafts=",".join(map(str, drafts)),
                    q_heads=hq, kv_heads=hkv, head_dim=head_dim, page=page, dtype=dtype)
    m = _log(rng, 1, 2048)
    n = 8 * (2 * _log(rng, 32, 14336 // 16) + rng.choice([-1, 1]))
    k = rng.choice([512, 640, 1024, 1408, 2048, 2560, 3584, 4096])
    return dict(op="linear", m=m, n=n, k=k, group=rng.choice([32, 64, 128, 128, 128]), sym=rng.random() < 0.3,
                act=rng.choice(ACTS), bias=rng.random() < 0.5, mul=rng.random() < 0.4,
                residual=rng.random() < 0.5)


def _ints(text):
    return [int(v) for v in text.split(",")]


def work(case):
    op = case["op"]
    if op == "linear":
        m, n, k, g = case["m"], case["n"], case["k"], case["group"]
        weights = n * k / 2 + n * (k // g) * (2.0 if case["sym"] else 2.5)
        io = 2 * m * k + 2 * k + 2 * m * n * (1 + case["mul"] + case["residual"]) + 2 * n * case["bias"]
        return {"bytes": weights + io, "flops": 2.0 * m * n * k}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op == "rope":
        tokens = sum(_ints(case["lengths"]))
        return {"bytes": 2.0 * 2 * tokens * (hq + 2 * hkv) * d + 12 * tokens,
                "flops": 3.0 * tokens * (hq + hkv) * case["rot_dim"]}
    if op == "prompt":
        lens = _ints(case["lengths"])
        return {"bytes": 2.0 * sum(lens) * (2 * hq + 2 * hkv) * d,
                "flops": 4.0 * d * hq * sum(n * (n + 1) / 2 for n in lens)}
    pairs = list(zip(_ints(case["contexts"]), _ints(case["drafts"])))
    return {"bytes": 2.0 * d * (2 * hkv * sum(c + t for c, t in pairs) + 2 * hq * sum(t for _, t in pairs)),
            "flops": 4.0 * d * hq * sum(t * (c + t) for c, t in pairs)}


# --------------------------------------------------------------------------- inputs

def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _heads_input(gen, tokens, heads, d, dtype):
    """Activations of a projection: ~N(0, 1), a few channels of each head larger."""
    gain = torch.ones(heads, d, device=DEV)
    gain[:, torch.randint(0, d, (max(1, d // 64),), generator=gen, device=DEV)] = 4.0
    return (_randn(gen, tokens, heads, d) * gain).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cumulative(lengths):
    total = [0]
    for n in lengths:
        total.append(total[-1] + n)
    return _i32(total)


def _pages(gen, lengths, page):
    """A block table with the pages of all sequences in random order, and the page count."""
    need = [(n + page - 1) // page for n in lengths]
    order = torch.randperm(sum(need) + 3, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(len(lengths), max(max(need), 1), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + 3


def _prepare_linear(case, gen):
    m, n, k, group, sym = case["m"], case["n"], case["k"], case["group"], case["sym"]
    sets = max(1, 128 // group)
    tiles, units = (n + 15) // 16, k // 128
    # the packed layout of awq_repack: codes, scales and zeros, each region 256-byte aligned
    nibbles = (8 + 2.5 * _randn(gen, tiles * units * 1024, 2)).round().clamp(0, 15).to(torch.uint8)
    codes = nibbles[:, 0] | (nibbles[:, 1] << 4)
    # groups wider than a unit repeat their set in each unit
    per = max(1, group // 128)
    scales = 0.008 * (0.5 + torch.rand(tiles, units // per, sets, 16, generator=gen, device=DEV))
    scales = scales.repeat_interleave(per, 1).to(torch.float16)
    zeros = torch.randint(6, 11, (tiles, units // per, sets, 8, 2), generator=gen, device=DEV).to(torch.uint8)
    zeros = zeros.repeat_interleave(per, 1)
    parts = [codes, scales.reshape(-1).view(torch.uint8)]
    if not sym:
        parts.append((zeros[..., 0] | (zeros[..., 1] << 4)).reshape(-1))
    padded = [torch.nn.functional.pad(p, (0, -p.numel() % 256)) for p in parts[1:]]
    packed = torch.cat([parts[0]] + padded)
    gain = torch.ones(k, device=DEV)
    gain[torch.randperm(k, generator=gen, device=DEV)[:max(1, k // 100)]] = 20.0
    s = dict(case=case, packed=packed, x=(_randn(gen, m, k) * gain).to(torch.float16),
             inv=(1.0 / gain.sqrt()).to(torch.float16), bias=None, mul=None, residual=None, ws=None)
    if case["bias"]:
        s["bias"] = _randn(gen, n, dtype=torch.float16)
    if case["mul"]:
        s["mul"] = _randn(gen, m, n, dtype=torch.float16)
    if case["residual"]:
        s["residual"] = _randn(gen, m, n, dtype=torch.float16)
    return s


def _prepare_rope(case, gen):
    lengths, dt = _ints(case["lengths"]), DTYPES[case["dtype"]]
    tokens, d, page, rot = sum(lengths), case["head_dim"], case["page"], case["rot_dim"]
    table, pages = _pages(gen, lengths, page)
    steps = torch.cat([torch.arange(n, device=DEV) for n in lengths])
    seq = torch.repeat_interleave(torch.arange(len(lengths), device=DEV), torch.tensor(lengths, device=DEV))
    base = 10000.0 if case["start"] < 8192 else 500000.0   # long contexts use a larger base
    freqs = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    cache = (pages, case["kv_heads"], page, d)
    return dict(case=case, q=_heads_input(gen, tokens, case["q_heads"], d, dt),
                k=_heads_input(gen, tokens, case["kv_heads"], d, dt),
                v=_randn(gen, tokens, case["kv_heads"], d, dtype=dt),
                positions=(steps + case["start"]).to(torch.int32), inv_freq=freqs.float().to(DEV),
                slots=(table[seq, steps // page].long() * page + steps % page),
                k_cache=_randn(gen, *cache, dtype=dt), v_cache=_randn(gen, *cache, dtype=dt))


def _prepare_prompt(case, gen):
    lengths, dt = _ints(case["lengths"]), DTYPES[case["dtype"]]
    tokens, hq, hkv, d = sum(lengths), case["q_heads"], case["kv_heads"], case["head_dim"]
    # one buffer of a fused q|k|v projection: the operands are strided views of it
    qkv = torch.cat([_heads_input(gen, tokens, hq + hkv, d, dt), _randn(gen, tokens, hkv, d, dtype=dt)], 1)
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                cu_seqlens=_cumulative(lengths), lengths=torch.tensor(lengths, device=DEV), most=max(lengths))


def _prepare_tree(case, gen):
    ctx, drafts, dt = _ints(case["contexts"]), _ints(case["drafts"]), DTYPES[case["dtype"]]
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    table, pages = _pages(gen, [c + t for c, t in zip(ctx, drafts)], page)
    pick = torch.rand(sum(drafts), generator=gen, device=DEV).tolist()
    mask, at = [], 0
    for t in drafts:   # a random tree: each token hangs on one of the few before it, or on the context
        bits = []
        for i in range(t):
            parent = i - 1 - int(4 * pick[at + i] ** 2)
            bits.append((bits[parent] if parent >= 0 else 0) | 1 << i)
        mask += [b - (1 << 64) if b >> 63 else b for b in bits]
        at += t
    cache = (pages, hkv, page, d)
    return dict(case=case, q=_heads_input(gen, sum(drafts), hq, d, dt), k_cache=_randn(gen, *cache, dtype=dt),
                v_cache=_randn(gen, *cache, dtype=dt), block_table=table, ctx_lens=_i32(ctx),
                cu_q=_cumulative(drafts), drafts=torch.tensor(drafts, device=DEV), max_q=max(drafts),
                mask=torch.tensor(mask, dtype=torch.int64, device=DEV))


_PREPARE = {"linear": _prepare_linear, "rope": _prepare_rope, "prompt": _prepare_prompt, "tree": _prepare_tree}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return _PREPARE[case["op"]](case, gen)


# ----------------------------------------------------------------------- plain forms

def _unpack(packed, n, k, group, sym):
    """W_d [n, k] as float32: the packed layout's codes, scales and zeros, and the binary16
    values binary16((q - z) * s) that the format defines."""
    sets, tiles, units = max(1, 128 // group), (n + 15) // 16, k // 128
    size = tiles * units * 1024
    words = packed[:size].view(torch.int32).view(tiles, units, 4, 16, 4)   # tile, unit, lane / 16, row, word
    # channel e of a word sits at nibble (e >> 1) + 4 (e & 1)
    shifts = torch.tensor([4 * ((e >> 1) + 4 * (e & 1)) for e in range(8)], dtype=torch.int32, device=DEV)
    q = ((words[..., None] >> shifts) & 15).float()                        # ..., word, channel
    which = torch.arange(4, device=DEV) * sets // 4                         # the set of each lane quarter
    scales = packed[size:size + tiles * units * sets * 32].view(torch.float16).view(tiles, units, sets, 16).float()
    s = scales[:, :, which]
    if sym:
        z = torch.full_like(s, 8.0)
    else:
        at = size + (tiles * units * sets * 32 + 255) // 256 * 256
        zb = packed[at:at + tiles * units * sets * 8].view(tiles, units, sets, 8, 1)
        z = torch.cat([zb & 15, zb >> 4], -1).view(tiles, units, sets, 16).float()[:, :, which]
    w = ((q - z[..., None, None]) * s[..., None, None]).half().float()
    return w.permute(0, 3, 1, 2, 4, 5).reshape(tiles * 16, k)[:n]


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


def _plain_linear(s):
    c = s["case"]
    x = (s["x"].float() * s["inv"].float()).half().float()   # X' is binary16 by definition
    y = x @ _unpack(s["packed"], c["n"], c["k"], c["group"], c["sym"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, c["act"])
    if s["mul"] is not None:
        y = y * s["mul"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.half()


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    xf = x.float()
    a, b = (xf[..., 0:rot:2], xf[..., 1:rot:2]) if interleaved else (xf[..., :rot // 2], xf[..., rot // 2:rot])
    first, second = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([first, second], -1).flatten(-2) if interleaved else torch.cat([first, second], -1)
    return torch.cat([turned, xf[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].float()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    page, offset = s["slots"] // c["page"], s["slots"] % c["page"]
    s["k_cache"][page, :, offset] = _rotate(s["k"], cos, sin, c["interleaved"])
    s["v_cache"][page, :, offset] = s["v"]
    return {"q": _rotate(s["q"], cos, sin, c["interleaved"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _softmax_product(scores, allowed, v):
    """softmax over the allowed columns times v; rows with none give zeros."""
    scores = scores.masked_fill(~allowed, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    return (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _padded(x, cu, lengths, most):
    """Packed [tokens, ...] to [sequences, most, ...], and the index that packs it again."""
    steps = torch.arange(most, device=DEV)
    real = steps < lengths[:, None]
    at = (cu[:-1, None].long() + steps).clamp_max(x.shape[0] - 1)
    return x[at], real


def _plain_prompt(s):
    c = s["case"]
    hkv, group = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    q, real = _padded(s["q"], s["cu_seqlens"], s["lengths"], s["most"])
    k, _ = _padded(s["k"], s["cu_seqlens"], s["lengths"], s["most"])
    v, _ = _padded(s["v"], s["cu_seqlens"], s["lengths"], s["most"])
    b, n, _, d = q.shape
    q = q.float().view(b, n, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * n, d)
    k, v = k.float().transpose(1, 2).contiguous(), v.float().transpose(1, 2).contiguous()
    scores = (q * d ** -0.5) @ k.transpose(-1, -2)
    steps = torch.arange(n, device=DEV)
    allowed = (steps[None, :] <= steps[:, None]).repeat(group, 1)
    out = _softmax_product(scores, allowed, v).view(b, hkv, group, n, d).permute(0, 3, 1, 2, 4)
    return out.reshape(b, n, hkv * group, d)[real].to(s["q"].dtype)


def _plain_tree(s):
    c = s["case"]
    hkv, group, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    q, real = _padded(s["q"], s["cu_q"], s["drafts"], s["max_q"])
    mask, _ = _padded(s["mask"], s["cu_q"], s["drafts"], s["max_q"])
    b, t = q.shape[:2]
    table = s["block_table"].long()
    k = s["k_cache"][table].float().transpose(1, 2).reshape(b, hkv, -1, d)
    v = s["v_cache"][table].float().transpose(1, 2).reshape(b, hkv, -1, d)
    q = q.float().view(b, t, hkv, group, d).transpose(1, 2).reshape(b, hkv, t * group, d)
    scores = (q * d ** -0.5) @ k.transpose(-1, -2)
    behind = torch.arange(k.shape[2], device=DEV) - s["ctx_lens"][:, None].long()   # < 0: in the context
    drafted = (mask[:, :, None] >> behind.clamp(0, 63)[:, None]) & 1
    allowed = (behind < 0)[:, None] | ((behind < s["drafts"][:, None])[:, None] & (drafted == 1))
    allowed = allowed[:, None, :, None].expand(b, 1, t, group, -1).reshape(b, 1, t * group, -1)
    out = _softmax_product(scores, allowed, v).view(b, hkv, t, group, d).transpose(1, 2)
    return out.reshape(b, t, hkv * group, d)[real].to(s["q"].dtype)


_PLAIN = {"linear": _plain_linear, "rope": _plain_rope, "prompt": _plain_prompt, "tree": _plain_tree}


# ------------------------------------------------------------- the package's operators

def _own_linear(s):
    from bit_weight_only_w4a16_amd import awq, block
    c = s["case"]
    ws = awq.workspace(c["m"], c["n"], c["k"], DEV, c["group"])
    return block.awq_gemm_fused(s["x"], s["inv"], s["packed"], c["n"], c["k"], c["group"], int(c["sym"]),
                                bias=s["bias"], act=c["act"], mul=s["mul"], residual=s["residual"], ws=ws)


def _own_rope(s):
    from bit_weight_only_w4a16_amd import block
    q, _ = block.awq_rope(s["q"], s["positions"], s["inv_freq"], k=s["k"], v=s["v"], k_cache=s["k_cache"],
                          v_cache=s["v_cache"], slots=s["slots"], interleaved=s["case"]["interleaved"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_prompt(s):
    from bit_weight_only_w4a16_amd import block
    return block.awq_attn_prompt(s["q"], s["k"], s["v"], s["cu_seqlens"])


def _own_tree(s):
    from bit_weight_only_w4a16_amd import block
    return block.awq_attn_tree(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["ctx_lens"], s["cu_q"],
                               s["max_q"], mask=s["mask"])


_OWN = {"linear": _own_linear, "rope": _own_rope, "prompt": _own_prompt, "tree": _own_tree}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ float64 definitions

def _exact_linear(s):
    c = s["case"]
    n, k, group, m = c["n"], c["k"], c["group"], c["m"]
    sets, units = max(1, 128 // group), k // 128
    tiles = (n + 15) // 16
    buf = s["packed"]
    scale_at = tiles * units * 1024
    zero_at = scale_at + (tiles * units * sets * 32 + 255) // 256 * 256
    scale_words = buf[scale_at:scale_at + tiles * units * sets * 32].view(torch.float16).double()
    kk = torch.arange(k, device=DEV)
    unit, quarter, word, e = kk // 128, kk % 128 // 32, kk % 32 // 8, kk % 8
    nibble = e // 2 + 4 * (e % 2)
    x = (s["x"].double() * s["inv"].double()).half().double()
    y = torch.empty(m, n, dtype=torch.float64, device=DEV)
    for r0 in range(0, n, 2048):
        rows = torch.arange(r0, min(n, r0 + 2048), device=DEV)[:, None]
        tile, r = rows // 16, rows % 16
        at = (tile * units + unit) * 1024 + (16 * quarter + r) * 16 + 4 * word + nibble // 2
        code = (buf[at].int() >> (4 * (nibble % 2)).int()) & 15
        block_set = (tile * units + unit) * sets + quarter * sets // 4
        scale = scale_words[block_set * 16 + r]
        if c["sym"]:
            zero = 8.0
        else:
            zero = ((buf[zero_at + block_set * 8 + r // 2].int() >> (4 * (r % 2)).int()) & 15).double()
        w = ((code.double() - zero) * scale).half().double()
        y[:, r0:r0 + 2048] = torch.mm(x, w.t().contiguous())
    if s["bias"] is not None:
        y += s["bias"].double()
    act = {"none": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
           "gelu": lambda t: t * 0.5 * torch.erfc(-t / math.sqrt(2.0)),
           "gelu_tanh": lambda t: t * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3))}
    y = act[c["act"]](y)
    if s["mul"] is not None:
        y *= s["mul"].double()
    if s["residual"] is not None:
        y += s["residual"].double()
    return y


def _exact_rope(s):
    c = s["case"]
    rot, half = c["rot_dim"], c["rot_dim"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotated(x):
        y = x.double().clone()
        first = slice(0, rot, 2) if c["interleaved"] else slice(0, half)
        second = slice(1, rot, 2) if c["interleaved"] else slice(half, rot)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    caches = {}
    for name, rows in (("k_cache", rotated(s["k"])), ("v_cache", s["v"].double())):
        flat = s[name].double().transpose(1, 2).reshape(-1, c["kv_heads"], c["head_dim"])
        flat[s["slots"]] = rows
        caches[name] = flat.view(-1, c["page"], c["kv_heads"], c["head_dim"]).transpose(1, 2).contiguous()
    return {"q": rotated(s["q"]), **caches}


def _exact_prompt(s):
    c = s["case"]
    group, d = c["q_heads"] // c["kv_heads"], c["head_dim"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for n in _ints(c["lengths"]):
        later = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
        for h in range(c["q_heads"]):
            k, v = s["k"][at:at + n, h // group].double(), s["v"][at:at + n, h // group].double().contiguous()
            w = torch.mm(s["q"][at:at + n, h].double(), k.t().contiguous()) / math.sqrt(d)
            out[at:at + n, h] = torch.mm(torch.softmax(w.masked_fill(later, -math.inf), 1), v)
        at += n
    return out


def _exact_tree(s):
    c = s["case"]
    group, d, page = c["q_heads"] // c["kv_heads"], c["head_dim"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (ctx, t) in enumerate(zip(_ints(c["contexts"]), _ints(c["drafts"]))):
        pages = s["block_table"][b, :(ctx + t + page - 1) // page].long()
        bits = (s["mask"][at:at + t, None] >> torch.arange(t, device=DEV)) & 1
        hidden = torch.cat([torch.zeros(t, ctx, dtype=torch.bool, device=DEV), bits == 0], 1)
        for h in range(c["kv_heads"]):
            k = s["k_cache"][pages, h].reshape(-1, d)[:ctx + t].double()
            v = s["v_cache"][pages, h].reshape(-1, d)[:ctx + t].double().contiguous()
            for g in range(h * group, (h + 1) * group):
                w = torch.mm(s["q"][at:at + t, g].double(), k.t().contiguous()) / math.sqrt(d)
                out[at:at + t, g] = torch.mm(torch.softmax(w.masked_fill(hidden, -math.inf), 1), v)
        at += t
    return out


_EXACT = {"linear": _exact_linear, "rope": _exact_rope, "prompt": _exact_prompt, "tree": _exact_tree}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
