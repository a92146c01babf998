"""The decoder-block operators on the GPU against plain float64 forms (block_ref), at the
sizes, layouts and masks where they can go wrong."""
import pytest

import block_ref as ref

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
block = pytest.importorskip("bit_weight_only_w4a16_amd.block")

pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16


def randn(*shape, seed, dtype=F16, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (gain * torch.randn(*shape, generator=g)).to(dtype)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def cumulative(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return i32(at)


# ------------------------------------------------------------------------ fused product

def layer(n, k, group, fmt, seed):
    w = randn(n, k, seed=seed, gain=0.05).to(DEV)
    s_c, inv = awq.awq_channel_scale(randn(32, k, seed=seed + 1).to(DEV), 0.5)
    qw, sc, qz = awq.awq_pack(w, s_c, group, fmt)
    packed = awq.awq_repack(qw, sc, qz, n, k, group, fmt)
    return packed, inv, awq.awq_dequant(packed, None, None, awq.LAYOUT_GFX950, n, k, group, fmt)


# M, N, K, group, fmt: decode kernel (one and more row tiles, sixteen wavefronts, exact and
# corrected), narrow tiles with and without a split of K, 65 <= M < 256, wide tiles with two,
# three and four column tiles and K split inside and across workgroups; ragged M and N
PRODUCTS = [
    (1, 72, 256, 128, 0), (2, 4104, 1024, 128, 1), (3, 264, 1024, 32, 0), (4, 4104, 8192, 128, 0),
    (5, 136, 512, 64, 1), (16, 4136, 512, 128, 0), (12, 4096, 11008, 128, 0), (17, 200, 1024, 128, 0),
    (33, 1032, 2048, 128, 1), (64, 520, 512, 256, 0), (100, 776, 2048, 128, 0), (255, 1544, 512, 64, 0),
    (256, 1032, 1024, 128, 0), (300, 2056, 512, 128, 1), (512, 11008, 512, 128, 0), (1100, 15368, 256, 128, 0),
    (2100, 6144, 256, 32, 1),
]


@pytest.mark.parametrize("m,n,k,group,fmt", PRODUCTS)
def test_fused_without_a_tail_is_the_plain_product(m, n, k, group, fmt):
    packed, inv, _ = layer(n, k, group, fmt, seed=m)
    x = randn(m, k, seed=m + 7).to(DEV)
    for ws in (awq.workspace(m, n, k, DEV, group), None):
        y0 = awq.awq_gemm(x, inv, packed, n, k, group, fmt, ws=ws)
        y1 = block.awq_gemm_fused(x, inv, packed, n, k, group, fmt, ws=ws)
        assert torch.equal(y0.view(torch.int16), y1.view(torch.int16))


@pytest.mark.parametrize("m,n,k,group,fmt", PRODUCTS)
@pytest.mark.parametrize("act,operands", [("none", "r"), ("silu", "m"), ("gelu", "bmr"), ("gelu_tanh", "br"),
                                          ("relu", "b")])
def test_fused_tail(m, n, k, group, fmt, act, operands):
    packed, inv, w_d = layer(n, k, group, fmt, seed=m + 100)
    x = randn(m, k, seed=m + 107).to(DEV)
    bias = randn(n, seed=1).to(DEV) if "b" in operands else None
    mul = randn(m, n, seed=2).to(DEV) if "m" in operands else None
    residual = randn(m, n, seed=3).to(DEV) if "r" in operands else None
    y = block.awq_gemm_fused(x, inv, packed, n, k, group, fmt, bias=bias, act=act, mul=mul, residual=residual,
                             ws=awq.workspace(m, n, k, DEV, group))
    rows = torch.unique(torch.tensor([0, m // 2, m - 1]))
    cols = torch.unique(torch.cat([torch.arange(0, min(n, 40)), torch.arange(n - 40, n)]).clamp_min(0))
    xs = (ref.cpu64(x[rows]) * ref.cpu64(inv)).half().double()
    v = xs @ ref.cpu64(w_d[cols]).t()
    # the product's documented accuracy: 2e-3 of its largest value
    pick = lambda t: None if t is None else t[rows][:, cols]  # noqa: E731
    want, bound = ref.tail(v, act, None if bias is None else bias[cols], pick(mul), pick(residual),
                           2e-3 * float(v.abs().max()))
    ref.check(y[rows][:, cols], want, bound, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1, 256, 512), (40, 264, 512), (300, 520, 512)])
def test_fused_in_place(m, n, k):
    packed, inv, _ = layer(n, k, 128, 0, seed=5)
    x, r = randn(m, k, seed=6).to(DEV), randn(m, n, seed=7).to(DEV)
    ws = awq.workspace(m, n, k, DEV)
    apart = block.awq_gemm_fused(x, inv, packed, n, k, residual=r, ws=ws)
    inside = r.clone()
    block.awq_gemm_fused(x, inv, packed, n, k, residual=inside, y=inside, ws=ws)
    assert torch.equal(apart, inside)
    apart = block.awq_gemm_fused(x, inv, packed, n, k, act="silu", mul=r, ws=ws)
    inside = r.clone()
    block.awq_gemm_fused(x, inv, packed, n, k, act="silu", mul=inside, y=inside, ws=ws)
    assert torch.equal(apart, inside)


def test_fused_extremes_of_the_activations():
    """Far negative and positive sums, and NaN: activations end at 0, at v, at NaN."""
    n, k = 128, 128
    packed, _, _ = layer(n, k, 128, 0, seed=8)
    x = torch.zeros(3, k, dtype=F16, device=DEV)
    bias = torch.tensor([-60000.0, 60000.0, -20.0, 20.0, -0.0, float("nan"), 5e-8, -1.0] * (n // 8),
                        dtype=F16, device=DEV)
    for act, f in ref.ACTS.items():
        y = block.awq_gemm_fused(x, None, packed, n, k, bias=bias, act=act)
        want = f(ref.cpu64(bias)).expand(3, n)
        ref.check(y, want, 2.0 ** -11 * want.abs() + 1e-6 * ref.cpu64(bias).abs().clamp_max(30).expand(3, n) + 2.0 ** -25,
                  act)


# ----------------------------------------------------------------------------- rotary

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 16), (80, 80), (80, 20), (72, 18), (72, 72), (8, 8),
                                   (96, 2), (40, 40)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_forms(dtype, d, rot, interleaved):
    tokens, hq, hkv = 37, 6, 3
    q, k = randn(tokens, hq, d, seed=1, dtype=dtype).to(DEV), randn(tokens, hkv, d, seed=2, dtype=dtype).to(DEV)
    pos = torch.randint(0, 131072, (tokens,), generator=torch.Generator().manual_seed(3)).to(torch.int32).to(DEV)
    freq, _ = block.rope_frequencies(rot, device=DEV)
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        qo, ko = block.awq_rope(q, pos, freq, k=k, interleaved=interleaved, inverse=inverse, scale=scale)
        for got, x in ((qo, q), (ko, k)):
            ref.check(got, *ref.rope(x, pos, freq, interleaved, inverse, scale), what=f"{d}/{rot}")


def test_rope_in_place_strided_and_q_or_k_alone():
    tokens, hq, hkv, d = 19, 4, 2, 64
    fused = randn(tokens, hq + 2 * hkv, d, seed=4).to(DEV)
    pos, (freq, _) = i32(list(range(tokens))), block.rope_frequencies(d, device=DEV)
    want_q, bound_q = ref.rope(fused[:, :hq], pos, freq)
    want_k, bound_k = ref.rope(fused[:, hq:hq + hkv], pos, freq)
    before = fused.clone()
    q, k = fused[:, :hq], fused[:, hq:hq + hkv]
    got, none = block.awq_rope(q, pos, freq)
    assert none is None
    ref.check(got, want_q, bound_q)
    none, got = block.awq_rope(None, pos, freq, k=k)
    assert none is None
    ref.check(got, want_k, bound_k)
    assert torch.equal(fused, before)
    block.awq_rope(q, pos, freq, k=k, q_out=q, k_out=k)
    ref.check(fused[:, :hq], want_q, bound_q)
    ref.check(fused[:, hq:hq + hkv], want_k, bound_k)
    assert torch.equal(fused[:, hq + hkv:], before[:, hq + hkv:])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("outer", ["heads", "slots"])
@pytest.mark.parametrize("d,rot,page", [(128, 128, 16), (80, 20, 5), (64, 32, 1)])
def test_rope_cache(dtype, outer, d, rot, page):
    """k and v reach their slots in either cache layout; slots of -1 and past the cache are not
    stored, and no other slot changes."""
    tokens, hq, hkv, pages = 23, 4, 2, 60 // page
    q, k, v = (randn(tokens, h, d, seed=s, dtype=dtype).to(DEV) for h, s in ((hq, 1), (hkv, 2), (hkv, 3)))
    kc, vc = (randn(*((pages, hkv, page, d) if outer == "heads" else (pages, page, hkv, d)), seed=s,
                    dtype=dtype).to(DEV) for s in (4, 5))
    if outer == "slots":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(6))[:tokens]
    slots[3], slots[7], slots[8] = -1, pages * page, 1 << 40
    pos, (freq, _) = i32(list(range(100, 100 + tokens))), block.rope_frequencies(rot, device=DEV)
    want_k, bound_k = ref.rope(k, pos, freq)
    at = [(i, int(s)) for i, s in enumerate(slots) if 0 <= int(s) < pages * page]
    expect_v, flat = vc.clone(), kc.clone()
    for i, s in at:
        expect_v[s // page, :, s % page] = v[i]
    qo, ko = block.awq_rope(q, pos, freq, k=k, v=v, k_cache=kc, v_cache=vc, slots=slots.to(DEV))
    assert ko is None
    ref.check(qo, *ref.rope(q, pos, freq))
    assert torch.equal(vc, expect_v)
    for i, s in at:
        ref.check(kc[s // page, :, s % page], want_k[i], bound_k[i])
        flat[s // page, :, s % page] = kc[s // page, :, s % page]
    assert torch.equal(kc, flat)
    kept = torch.empty_like(k)
    block.awq_rope(q, pos, freq, k=k, v=v, k_cache=kc, v_cache=vc, slots=slots.to(DEV), k_out=kept)
    ref.check(kept, want_k, bound_k)


def test_rope_v_is_copied_bit_for_bit():
    """Infinities and NaN in v reach the cache as they are; so do q's elements past rot_dim."""
    tokens, d, page = 5, 64, 4
    v = randn(tokens, 1, d, seed=1)
    v[0, 0, 0], v[1, 0, 1], v[2, 0, 40] = float("inf"), float("-inf"), float("nan")
    q = v.clone()
    kc, vc = (torch.zeros(2, 1, page, d, dtype=F16, device=DEV) for _ in range(2))
    freq, _ = block.rope_frequencies(16, device=DEV)
    qo, _ = block.awq_rope(q.to(DEV), i32([0] * tokens), freq, k=torch.zeros(tokens, 1, d, dtype=F16, device=DEV),
                           v=v.to(DEV), k_cache=kc, v_cache=vc, slots=torch.arange(tokens, device=DEV))
    got = vc.transpose(1, 2).reshape(-1, 1, d)[:tokens].cpu()
    assert torch.equal(got.view(torch.int16), v.view(torch.int16))
    assert torch.equal(qo.cpu().view(torch.int16)[..., 16:], q.view(torch.int16)[..., 16:])


# ---------------------------------------------------------------------- prompt attention

def prompt_inputs(lengths, hq, hkv, d, dtype, seed, spare=0):
    n = sum(lengths) + spare
    qkv = randn(n, hq + 2 * hkv, d, seed=seed, dtype=dtype, gain=1.5)
    return qkv, n


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lengths", [[1], [2, 1, 0, 3], [31, 32, 33], [63, 64, 65, 0], [127, 128, 129], [200, 1, 300]])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (6, 2, 64)])
def test_prompt_lengths(dtype, lengths, hq, hkv, d):
    qkv, _ = prompt_inputs(lengths, hq, hkv, d, dtype, seed=sum(lengths))
    q, k, v = qkv.to(DEV).split([hq, hkv, hkv], 1)
    out = block.awq_attn_prompt(q, k, v, cumulative(lengths))
    ref.check(out, *ref.prompt(q, k, v, lengths))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 80, 96, 120, 128])
def test_prompt_head_sizes(dtype, d):
    lengths = [70, 141]
    qkv, _ = prompt_inputs(lengths, 3, 1, d, dtype, seed=d)
    q, k, v = qkv.to(DEV).split([3, 1, 1], 1)
    out = block.awq_attn_prompt(q, k, v, cumulative(lengths), scale=0.3)
    ref.check(out, *ref.prompt(q, k, v, lengths, scale=0.3))


def test_prompt_layouts_and_rows_outside():
    """Heads outermost, an output with a gap between tokens, and tokens in no sequence (not
    written)."""
    lengths, hq, hkv, d = [50, 90], 4, 2, 64
    qkv, n = prompt_inputs(lengths, hq, hkv, d, F16, seed=9, spare=7)
    q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in qkv.to(DEV).split([hq, hkv, hkv], 1))
    wide = torch.full((n, hq + 3, d), 7.0, dtype=F16, device=DEV)
    out = wide[:, 1:1 + hq]
    block.awq_attn_prompt(q, k, v, cumulative(lengths), out=out)
    want, bound = ref.prompt(q, k, v, lengths)
    ref.check(out[:140], want[:140], bound[:140])
    assert bool((wide[140:] == 7).all() and (wide[:, 0] == 7).all() and (wide[:, 1 + hq:] == 7).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_prompt_later_tokens_never_reach_a_row(dtype, bad):
    """Infinities and NaN in a later token's key and value, and in the neighbouring sequence."""
    lengths, hq, hkv, d = [100, 150, 40], 2, 1, 128
    qkv, _ = prompt_inputs(lengths, hq, hkv, d, dtype, seed=11)
    qkv[:100, hq:] = bad           # the whole first sequence
    qkv[100 + 77:250, hq:] = bad   # the second from its token 77 on
    q, k, v = qkv.to(DEV).split([hq, hkv, hkv], 1)
    out = block.awq_attn_prompt(q, k, v, cumulative(lengths))
    rows = list(range(100, 177)) + list(range(250, 290))
    clean = qkv.clone()
    clean[:100, hq:] = 0
    clean[177:250, hq:] = 0
    want, bound = ref.prompt(*clean.split([hq, hkv, hkv], 1), lengths)
    ref.check(out[rows], want[rows], bound[rows])
    if bad != bad:  # and a token that is NaN itself stays NaN
        assert bool(torch.isnan(out[177:250]).all())


def test_prompt_large_scores():
    """Rows whose maximum moves far from key to key (the running maximum is rescaled often),
    and values near the type's largest."""
    lengths, d = [400], 64
    g = torch.Generator().manual_seed(13)
    q = torch.randn(400, 1, d, generator=g) * 6
    k = torch.randn(400, 1, d, generator=g) * torch.linspace(0.1, 8, 400)[:, None, None]
    v = torch.randn(400, 1, d, generator=g) * 15000
    q, k, v = (t.clamp(-60000, 60000).to(F16).to(DEV) for t in (q, k, v))
    out = block.awq_attn_prompt(q, k, v, cumulative(lengths))
    ref.check(out, *ref.prompt(q, k, v, lengths))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_scores_of_minus_infinity_first(dtype):
    """Rows whose first tiles hold only scores of -inf, then finite ones far below 0."""
    n, d = 300, 64
    g = torch.Generator().manual_seed(21)
    q = torch.rand(n, 1, d, generator=g) + 0.5
    k = -20 * (torch.rand(n, 1, d, generator=g) + 0.5)
    k[:150, 0, 3] = float("-inf")
    v = torch.randn(n, 1, d, generator=g)
    q, k, v = (t.to(dtype).to(DEV) for t in (q, k, v))
    out = block.awq_attn_prompt(q, k, v, cumulative([n]))
    # (keys of -inf have probability 0: the reference's rows past them leave them out)
    for t in (150, 151, 200, 299):
        sees = (torch.arange(n) >= 150)[None] & (torch.arange(n) <= t)[None]
        finite = torch.where(torch.isinf(k), torch.zeros_like(k), k)
        want, bound = ref.attend(ref.cpu64(q[t:t + 1, 0]), ref.cpu64(finite[:, 0]), ref.cpu64(v[:, 0]), sees, d ** -0.5,
                                 dtype)
        ref.check(out[t:t + 1, 0], want, bound, f"row {t}")


def test_prompt_many_sequences():
    """More sequences than a wavefront has lanes, empty ones among them."""
    lengths = [(i * 7) % 11 for i in range(150)]
    qkv, _ = prompt_inputs(lengths, 2, 2, 64, F16, seed=14)
    q, k, v = qkv.to(DEV).split([2, 2, 2], 1)
    out = block.awq_attn_prompt(q, k, v, cumulative(lengths))
    ref.check(out, *ref.prompt(q, k, v, lengths))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("count,hq,hkv", [(300, 8, 2), (140, 12, 3), (300, 2, 1), (5000, 4, 1)])
def test_prompt_batches_of_short_sequences(dtype, count, hq, hkv):
    """Several heads of a group in one workgroup; lengths of 0 to 70 tokens, one of 200. The
    largest batch is checked at a few sequences."""
    g = torch.Generator().manual_seed(count + hq)
    lengths = torch.randint(0, 71 if count < 1000 else 9, (count,), generator=g).tolist()
    lengths[count // 2] = 200
    qkv, _ = prompt_inputs(lengths, hq, hkv, 64, dtype, seed=count)
    q, k, v = qkv.to(DEV).split([hq, hkv, hkv], 1)
    out = block.awq_attn_prompt(q, k, v, cumulative(lengths))
    assert not bool(torch.isnan(out).any())
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    for b in {0, 1, 63, 64, 65, count // 2, count // 2 + 1, count - 2, count - 1}:
        at = slice(starts[b], starts[b + 1])
        ref.check(out[at], *ref.prompt(q[at], k[at], v[at], [lengths[b]]), f"sequence {b} of {lengths[b]}")


def test_prompt_long():
    """A few rows of a long sequence against float64 on the device."""
    n, hq, hkv, d = 5000, 8, 2, 128
    qkv = randn(n, hq + 2 * hkv, d, seed=15).to(DEV)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    out = block.awq_attn_prompt(q, k, v, cumulative([n]))
    for t in (0, 127, 128, 2047, 4095, 4999):
        for h in (0, 5):
            sees = torch.ones(1, t + 1, dtype=torch.bool)
            g = h // (hq // hkv)
            want, bound = ref.attend(ref.cpu64(q[t:t + 1, h]), ref.cpu64(k[:t + 1, g]), ref.cpu64(v[:t + 1, g]), sees,
                                     d ** -0.5, F16)
            ref.check(out[t:t + 1, h], want, bound, f"row {t} head {h}")


# ------------------------------------------------------------------------- tree attention

def tree_inputs(ctx, drafts, hq, hkv, d, page, dtype, seed, outer="heads", fill=float("nan")):
    """A cache with the sequences' pages in random order; everything else in it is `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [(c + t + page - 1) // page for c, t in zip(ctx, drafts)]
    order = torch.randperm(sum(need) + 2, generator=g)
    width = max(max(need), 1) + 1
    table = torch.full((len(ctx), width), 1 << 30, dtype=torch.int32)   # entries past a length are garbage
    table[:, -1] = -5
    shape = (sum(need) + 2, hkv, page, d) if outer == "heads" else (sum(need) + 2, page, hkv, d)
    kc, vc = (torch.full(shape, fill, dtype=dtype) for _ in range(2))
    if outer == "slots":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
        for cache in (kc, vc):
            x = torch.randn(hkv, ctx[b] + drafts[b], d, generator=g).to(dtype)
            for i in range(n):
                part = x[:, i * page:(i + 1) * page]
                cache[int(table[b, i]), :, :part.shape[1]] = part
    q = torch.randn(sum(drafts), hq, d, generator=g).to(dtype) * 1.5
    return q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV)


def words(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)


def tree_masks(drafts, seed):
    g = torch.Generator().manual_seed(seed)
    out = []
    for t in drafts:
        bits = []
        for i in range(t):
            p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        out += bits
    return out


def run_tree(ctx, drafts, hq, hkv, d, page, dtype, seed, masks="tree", outer="heads", **kw):
    q, kc, vc, table = tree_inputs(ctx, drafts, hq, hkv, d, page, dtype, seed, outer)
    masks = tree_masks(drafts, seed + 1) if masks == "tree" else masks
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), max(max(drafts), 1),
                              mask=None if masks is None else words(masks), **kw)
    want, bound = ref.tree(q, kc, vc, table, ctx, drafts, masks, kw.get("scale"))
    ref.check(out, want, bound)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("ctx", [[0], [1], [31, 32, 33], [127, 128, 129, 0], [700, 5, 0, 260]])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (8, 1, 64)])
def test_tree_single_tokens(dtype, ctx, hq, hkv, d):
    run_tree(ctx, [1] * len(ctx), hq, hkv, d, 16, dtype, seed=sum(ctx))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("ctx,drafts", [([0, 64, 13], [7, 1, 30]), ([77, 100, 0, 250], [64, 3, 64, 17]),
                                        ([32, 95, 96], [33, 0, 2])])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (12, 4, 64), (8, 1, 128)])
def test_tree_drafts(dtype, ctx, drafts, hq, hkv, d):
    run_tree(ctx, drafts, hq, hkv, d, 8, dtype, seed=len(ctx))
    run_tree(ctx, drafts, hq, hkv, d, 8, dtype, seed=len(ctx), masks=None)


@pytest.mark.parametrize("page", [1, 3, 8, 33, 64, 256])
@pytest.mark.parametrize("outer", ["heads", "slots"])
def test_tree_pages(page, outer):
    run_tree([150, 0, 61], [5, 2, 9], 4, 2, 64, page, F16, seed=page, outer=outer)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [8, 40, 72, 80, 96, 120])
def test_tree_head_sizes(dtype, d):
    run_tree([90, 33], [3, 20], 6, 2, d, 16, dtype, seed=d, scale=0.2)


def test_tree_rows_that_see_nothing():
    """No context and an empty mask: zeros, beside rows that see something, in one and in many
    splits."""
    for extra in (0, 1500):
        ctx, drafts = [0, 40, 0, extra], [4, 3, 1, 2]
        masks = [0, 2, 0, 9] + [0, 1, 7] + [0] + [0, 0]
        run_tree(ctx, drafts, 4, 2, 128, 16, F16, seed=21, masks=masks)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tree_masked_tokens_never_reach_a_row(dtype, bad):
    """Infinities and NaN in drafted tokens that some rows see and others do not."""
    ctx, drafts, hq, hkv, d, page = [45, 0], [6, 6], 4, 2, 128, 16
    q, kc, vc, table = tree_inputs(ctx, drafts, hq, hkv, d, page, dtype, seed=31)
    masks = [1, 3, 5, 11, 16, 33] * 2          # token 2's bit only in rows 2; token 4 alone
    clean_k, clean_v = kc.clone(), vc.clone()
    for b, c in enumerate(ctx):
        for j in (2, 4):
            pos = c + j
            pg = int(table[b, pos // page])
            kc[pg, :, pos % page], vc[pg, :, pos % page] = bad, bad
            clean_k[pg, :, pos % page], clean_v[pg, :, pos % page] = 0, 0
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), 6, mask=words(masks))
    want, bound = ref.tree(q, clean_k, clean_v, table, ctx, drafts, masks)
    rows = [0, 1, 3, 5, 6, 7, 9, 11]
    ref.check(out[rows], want[rows], bound[rows])
    if bad != bad:
        assert bool(torch.isnan(out[[2, 4, 8, 10]]).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("count,hq,hkv,d,longest", [(140, 4, 2, 128, 60), (270, 2, 1, 72, 300), (300, 2, 2, 64, 40)])
def test_tree_batches_of_many_sequences(dtype, count, hq, hkv, d, longest):
    """More workgroups than run at once, with a few rows each; empty sequences among them."""
    g = torch.Generator().manual_seed(count)
    ctx = torch.randint(0, longest, (count,), generator=g).tolist()
    drafts = torch.randint(0, 4, (count,), generator=g).tolist()
    run_tree(ctx, drafts, hq, hkv, d, 16, dtype, seed=count)


def test_tree_many_splits():
    """One sequence over a wide table of single-position pages: more splits than a wavefront
    has lanes, most of them empty for the short sequence beside it."""
    width, hkv, d = 60000, 1, 64
    ctx, drafts = [59000, 30], [1, 1]
    g = torch.Generator().manual_seed(41)
    table = torch.randperm(width, generator=g).to(torch.int32).repeat(2, 1).to(DEV)
    kc, vc = (torch.randn(width, hkv, 1, d, generator=g).to(F16).to(DEV) for _ in range(2))
    q = torch.randn(2, 4, d, generator=g).to(F16).to(DEV)
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), 1)
    ref.check(out, *ref.tree(q, kc, vc, table, ctx, drafts, None))


def test_tree_offsets_past_32_bits():
    """Pages whose elements start past 2^32 (a cache of 2^32 + elements per tensor)."""
    hkv, page, d = 8, 16, 128
    pages = (1 << 32) // (hkv * page * d) + 64
    kc, vc = (torch.empty(pages, hkv, page, d, dtype=F16, device=DEV) for _ in range(2))
    ctx, drafts = [100], [3]
    used = [pages - 1, 5, pages - 3, pages - 30, 0, pages - 2, 2]
    g = torch.Generator().manual_seed(51)
    small = []
    for cache in (kc, vc):
        x = torch.randn(7, hkv, page, d, generator=g).to(F16)
        cache[used] = x.to(DEV)
        small.append(x)
    q = torch.randn(3, 16, d, generator=g).to(F16).to(DEV)
    out = block.awq_attn_tree(q, kc, vc, i32([used]), i32(ctx), cumulative(drafts), 3)
    ref.check(out, *ref.tree(q, small[0], small[1], torch.arange(7)[None], ctx, drafts, None))
    # and the rotary write into such a page
    k, v = (torch.randn(2, hkv, d, generator=g).to(F16).to(DEV) for _ in range(2))
    slots = torch.tensor([(pages - 1) * page + 3, (pages - 40) * page], device=DEV)
    freq, _ = block.rope_frequencies(d, device=DEV)
    block.awq_rope(k, i32([5, 6]), freq, k=k, v=v, k_cache=kc, v_cache=vc, slots=slots)
    assert torch.equal(vc[pages - 1, :, 3], v[0]) and torch.equal(vc[pages - 40, :, 0], v[1])


def test_rope_of_more_threads_than_a_launch_has_along_x():
    """2^31 + threads: tokens of 16 elements, rotated by pairs of single elements."""
    n, d = (1 << 31) // 15 + 1000, 16
    x = torch.zeros(n, 1, d, dtype=F16, device=DEV)
    x[-5:] = 1.0
    positions = torch.zeros(n, dtype=torch.int32, device=DEV)
    freq = torch.tensor([1.0], device=DEV)
    positions[-5:] = i32([0, 1, 2, 3, 4])
    block.awq_rope(x, positions, freq, q_out=x)
    ref.check(x[-5:], *ref.rope(torch.ones(5, 1, d, dtype=F16), positions[-5:], freq))
    assert float(x[:-5].abs().max()) == 0.0


def test_tree_lengths_past_the_table_are_clamped():
    """A length that the table does not hold reads what the table holds, and no more."""
    hkv, page, d = 1, 16, 64
    q, kc, vc, table = tree_inputs([64], [0], 1, hkv, d, page, F16, seed=61, fill=0.0)
    q = torch.randn(1, 1, d, generator=torch.Generator().manual_seed(1)).to(F16).to(DEV)
    table = table[:, :4].contiguous()
    out = block.awq_attn_tree(q, kc, vc, table, i32([100000]), i32([0, 1]), 1)
    want, bound = ref.tree(q, kc, vc, table, [64], [1], [0])
    ref.check(out, want, bound)


# ------------------------------------------------------------------- streams and graphs

def test_another_stream_and_a_graph():
    """Calls on a side stream, and a captured decode step replayed with the program's own work
    between, give the eager results' bits."""
    ctx, drafts, hq, hkv, d, page = [300, 41], [2, 5], 8, 2, 128, 16
    q, kc, vc, table = tree_inputs(ctx, drafts, hq, hkv, d, page, F16, seed=71, fill=0.0)
    masks = words(tree_masks(drafts, 3))
    args = (q, kc, vc, table, i32(ctx), cumulative(drafts), 5)
    ws = torch.empty(max(1, block.awq_attn_tree_workspace_bytes(7, 2, table.shape[1], page, 5, hq, hkv, d)),
                     dtype=torch.uint8, device=DEV)
    freq, _ = block.rope_frequencies(d, device=DEV)
    pos = i32(list(range(7)))
    n, k = 256, hq * d
    packed, inv, _ = layer(n, k, 128, 0, seed=9)

    def step():
        turned, _ = block.awq_rope(q, pos, freq)
        a = block.awq_attn_tree(turned, *args[1:], mask=masks, ws=ws)
        y = block.awq_gemm_fused(a.view(7, k), inv, packed, n, k, act="silu")
        z = block.awq_attn_prompt(turned, kc.view(-1, hkv, d)[:7], vc.view(-1, hkv, d)[:7], i_cu)
        return y, z

    i_cu = i32([0, 3, 7])
    eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(3):
        for t in captured:
            t.zero_()
        torch.randn(1000, device=DEV).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b), i
        for a, b in zip(eager, step()):
            assert torch.equal(a, b), i


def test_a_graph_keeps_its_workspace():
    """A call that grows the stream's workspace after a graph was captured with the smaller
    one: what is allocated then is not what the graph writes to."""
    stream = torch.cuda.Stream()
    small, large = (tree_inputs([n], [t], 8, 1, 128, 16, F16, seed=n) for n, t in ((4000, 1), (9000, 40)))

    need = [block.awq_attn_tree_workspace_bytes(t, 1, x[3].shape[1], 16, t, 8, 1, 128) for x, t in ((small, 1), (large, 40))]
    assert 0 < need[0] < (1 << 20) < need[1]
    with torch.cuda.stream(stream):
        n1, cu1, n2, cu2 = i32([4000]), cumulative([1]), i32([9000]), cumulative([40])
        want = block.awq_attn_tree(*small, n1, cu1, 1)
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = block.awq_attn_tree(*small, n1, cu1, 1)
        block.awq_attn_tree(*large, n2, cu2, 40)
        others = [torch.full((1 << 20,), 77, dtype=torch.uint8, device=DEV) for _ in range(8)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            stream.synchronize()
            assert torch.equal(out, want)
            assert all(bool((x == 77).all()) for x in others)



# ---------------------------------------------------------------------------- refusals

def test_binding_refusals():
    """Types, shapes, layouts and devices that do not fit are errors, and nothing runs."""
    q = torch.zeros(4, 4, 64, dtype=F16, device=DEV)
    k = torch.zeros(4, 2, 64, dtype=F16, device=DEV)
    cu, pos = i32([0, 4]), i32([0, 1, 2, 3])
    freq = torch.ones(32, device=DEV)
    kc = torch.zeros(3, 2, 16, 64, dtype=F16, device=DEV)
    slots = torch.arange(4, device=DEV)
    prompt = block.awq_attn_prompt
    rope = block.awq_rope
    tree = block.awq_attn_tree
    good = (q, kc, kc.clone(), i32([[0, 1]]), i32([3]), i32([0, 4]), 4)
    tree(*good)

    def change(i, t):
        return good[:i] + (t,) + good[i + 1:]

    for error, fn in [
        (TypeError, lambda: prompt(q.float(), k, k, cu)),
        (TypeError, lambda: prompt(q, k.bfloat16(), k, cu)),
        (TypeError, lambda: prompt(q, k, k, cu.long())),
        (TypeError, lambda: prompt(q, k, k, None)),
        (ValueError, lambda: prompt(q, k[:3], k, cu)),
        (ValueError, lambda: prompt(q, k, k[:, :1], cu)),
        (ValueError, lambda: prompt(q[0], k, k, cu)),
        (ValueError, lambda: prompt(q, k.transpose(1, 2), k, cu)),
        (ValueError, lambda: prompt(q, k, k, cu[:0])),
        (ValueError, lambda: prompt(q, k, k, cu.cpu())),
        (ValueError, lambda: prompt(q, k, k, cu, out=q[:3])),
        (TypeError, lambda: prompt(q, k, k, cu, out=q.float())),
        (TypeError, lambda: prompt(q, k, k, cu, scale="x")),
        (awq.AwqError, lambda: prompt(q, k, k, cu, scale=0.0)),
        (awq.AwqError, lambda: prompt(q[:, :3], k, k, cu)),
        (ValueError, lambda: rope(None, pos, freq)),
        (ValueError, lambda: rope(q, pos[:3], freq)),
        (TypeError, lambda: rope(q, pos.long(), freq)),
        (TypeError, lambda: rope(q, pos, freq.double())),
        (ValueError, lambda: rope(q, pos, torch.ones(33, device=DEV))),
        (ValueError, lambda: rope(q, pos, freq, k=k[:2])),
        (ValueError, lambda: rope(q, pos, freq, k_out=k)),
        (ValueError, lambda: rope(q, pos, freq, k=k, v=k, k_cache=kc, slots=slots)),
        (ValueError, lambda: rope(q, pos, freq, k=k, k_cache=kc, v_cache=kc, slots=slots)),
        (ValueError, lambda: rope(q, pos, freq, k=k, v=k, k_cache=kc, v_cache=kc)),
        (TypeError, lambda: rope(q, pos, freq, k=k, v=k, k_cache=kc, v_cache=kc, slots=slots.int())),
        (ValueError, lambda: rope(q, pos, freq, k=k, v=k, k_cache=kc, v_cache=kc[:2], slots=slots)),
        (ValueError, lambda: rope(q, pos, freq, k=k, v=k, k_cache=kc[:, :1], v_cache=kc[:, :1], slots=slots)),
        (TypeError, lambda: rope(q, pos, freq, k=k, v=k, k_cache=kc.float(), v_cache=kc.float(), slots=slots)),
        (TypeError, lambda: tree(*change(0, q.float()))),
        (ValueError, lambda: tree(*change(1, kc[0]))),
        (ValueError, lambda: tree(*change(2, kc.transpose(0, 1)))),
        (ValueError, lambda: tree(*change(3, i32([0, 1])))),
        (ValueError, lambda: tree(*change(4, i32([3, 3])))),
        (ValueError, lambda: tree(*change(5, i32([0, 4, 4])))),
        (TypeError, lambda: tree(*change(6, None))),
        (awq.AwqError, lambda: tree(*change(6, 65))),
        (awq.AwqError, lambda: tree(*change(6, 0))),
        (ValueError, lambda: tree(*good, mask=torch.zeros(3, dtype=torch.int64, device=DEV))),
        (TypeError, lambda: tree(*good, mask=pos)),
        (TypeError, lambda: tree(*good, ws=pos)),
        (awq.AwqError, lambda: tree(q, kc, kc, torch.zeros(1, 500, dtype=torch.int32, device=DEV), *good[4:],
                                    ws=torch.zeros(16, dtype=torch.uint8, device=DEV))),
    ]:
        with pytest.raises(error):
            fn()
    n, kk = 128, 256
    packed, inv, _ = layer(n, kk, 128, 0, seed=1)
    x = torch.zeros(3, kk, dtype=F16, device=DEV)
    y = torch.zeros(3, n, dtype=F16, device=DEV)
    fused = block.awq_gemm_fused
    fused(x, inv, packed, n, kk, bias=y[0], mul=y, residual=y)
    for error, fn in [
        (ValueError, lambda: fused(x, inv, packed[:100], n, kk)),
        (TypeError, lambda: fused(x.float(), inv, packed, n, kk)),
        (ValueError, lambda: fused(x[:, :128], inv, packed, n, kk)),
        (ValueError, lambda: fused(x, inv[:128], packed, n, kk)),
        (ValueError, lambda: fused(x, inv, packed, n, kk, bias=y)),
        (ValueError, lambda: fused(x, inv, packed, n, kk, mul=y[:2])),
        (TypeError, lambda: fused(x, inv, packed, n, kk, residual=y.float())),
        (ValueError, lambda: fused(x, inv, packed, n, kk, y=y.t())),
        (ValueError, lambda: fused(x, inv, packed, n, kk, act="tanh")),
        (awq.AwqError, lambda: fused(x[:, :200].contiguous(), None, packed, n, 200)),
    ]:
        with pytest.raises(error):
            fn()
    torch.cuda.synchronize()


def test_calls_of_nothing():
    q = torch.zeros(0, 4, 64, dtype=F16, device=DEV)
    cu = i32([0])
    assert block.awq_attn_prompt(q, q[:, :2], q[:, :2], cu).shape == (0, 4, 64)
    assert block.awq_rope(q, i32([]), torch.ones(32, device=DEV))[0].shape == (0, 4, 64)
    kc = torch.zeros(1, 2, 16, 64, dtype=F16, device=DEV)
    assert block.awq_attn_tree(q, kc, kc, torch.zeros(1, 1, dtype=torch.int32, device=DEV), i32([0]), i32([0, 0]),
                               1).shape == (0, 4, 64)
    packed, inv, _ = layer(128, 128, 128, 0, seed=1)
    assert block.awq_gemm_fused(torch.zeros(0, 128, dtype=F16, device=DEV), inv, packed, 128, 128).shape == (0, 128)
