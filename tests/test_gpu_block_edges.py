"""Attention of the decoder block at its edges: what masked and visible infinities and NaN do
where a context is split over workgroups and elsewhere, values at the ends of the type's range,
and how long such inputs take."""
import pytest

import block_ref as ref

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
block = pytest.importorskip("bit_weight_only_w4a16_amd.block")

from test_gpu_block import DEV, cumulative, i32, randn, tree_inputs, tree_masks, words  # noqa: E402

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def splits(q, kc, table, max_q):
    """Partial results per row of such a call (1: none are kept)."""
    hkv, page, d = kc.shape[1:]
    need = block.awq_attn_tree_workspace_bytes(q.shape[0], table.shape[0], table.shape[1], page, max_q, q.shape[1], hkv,
                                               d)
    return max(1, need // (q.shape[0] * q.shape[1] * (d + 2) * 4))


def at(table, b, pos, page):
    return int(table[b, pos // page]), slice(None), pos % page


# ------------------------------------------------- infinities and NaN in split contexts

@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("drafts,hq,hkv", [([6, 6], 4, 2), ([6, 6], 8, 1), ([40, 33], 4, 2)])
def test_masked_tokens_never_reach_a_row_of_a_split_context(dtype, bad, drafts, hq, hkv):
    """Drafted tokens that most rows do not see hold infinities and NaN, and the context before
    them is in other splits (up to 16 rows, and more: both kernels)."""
    ctx, d, page = [3000, 700], 128, 16
    q, kc, vc, table = tree_inputs(ctx, drafts, hq, hkv, d, page, dtype, seed=32)
    assert splits(q, kc, table, max(drafts)) > 1
    masks = [m & ~0b10100 | 1 << t for n in drafts for t, m in enumerate(tree_masks([n], 33))]  # 2 and 4: by themselves
    clean_k, clean_v = kc.clone(), vc.clone()
    for b, c in enumerate(ctx):
        for j in (2, 4):
            i = at(table, b, c + j, page)
            kc[i], vc[i] = bad, bad
            clean_k[i], clean_v[i] = 0, 0
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), max(drafts), mask=words(masks))
    want, bound = ref.tree(q, clean_k, clean_v, table, ctx, drafts, masks)
    starts = [0, drafts[0]]
    rows = [s + t for s, n in zip(starts, drafts) for t in range(n) if t not in (2, 4)]
    ref.check(out[rows], want[rows], bound[rows])
    if bad != bad:
        assert bool(torch.isnan(out[[s + t for s in starts for t in (2, 4)]]).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("drafts,hq,hkv", [([1, 1], 4, 2), ([6, 6], 8, 1)])
def test_a_visible_nan_stays_in_its_channel(dtype, drafts, hq, hkv):
    """One channel of a visible value row is NaN, in the middle of a split context and among the
    new tokens: that channel is NaN, the others are right."""
    ctx, d, page = [3000, 700], 128, 16
    q, kc, vc, table = tree_inputs(ctx, drafts, hq, hkv, d, page, dtype, seed=34)
    assert splits(q, kc, table, max(drafts)) > 1
    for b, pos, channel in ((0, 1500, 5), (0, 3000, 70), (1, 3, 64)):
        vc[at(table, b, pos, page) + (channel,)] = float("nan")
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), max(drafts))
    want, bound = ref.tree(q, kc, vc, table, ctx, drafts, None)
    assert int(torch.isnan(want).sum()) == hq * (2 * drafts[0] + drafts[1])
    ref.check(out, want, bound)


# ---------------------------------------------------- strides of dimensions of one element

def test_one_token_of_a_long_tensor():
    """The last token of a prompt, as a model's decode takes it: its token stride is that of the
    whole prompt, and is not one of the call's."""
    q, k, v = (randn(1, 1100, h, 128, seed=s).to(DEV)[:, -1] for s, h in enumerate((64, 8, 8)))
    assert q.stride(0) > 1 << 23
    freq, _ = block.rope_frequencies(128, device=DEV)
    got_q, got_k = block.awq_rope(q, i32([77]), freq, k=k)
    ref.check(got_q, *ref.rope(q, i32([77]), freq))
    ref.check(got_k, *ref.rope(k, i32([77]), freq))
    ref.check(block.awq_attn_prompt(q, k, v, cumulative([1])), *ref.prompt(q, k, v, [1]))
    into = torch.zeros(1, 1100, 64, 128, dtype=F16, device=DEV)
    block.awq_attn_prompt(q, k, v, cumulative([1]), out=into[:, 5])
    ref.check(into[:, 5], *ref.prompt(q, k, v, [1]))
    assert float(into[:, :5].abs().max()) == 0.0 and float(into[:, 6:].abs().max()) == 0.0
    _, kc, vc, table = tree_inputs([50], [1], 64, 8, 128, 16, F16, 3)
    out = block.awq_attn_tree(q, kc, vc, table, i32([50]), cumulative([1]), 1)
    ref.check(out, *ref.tree(q, kc, vc, table, [50], [1], None))


@pytest.mark.parametrize("pages,hkv,page", [(40, 1, 1), (40, 2, 1), (5, 1, 8), (1, 1, 40), (1, 2, 40)])
def test_caches_with_dimensions_of_one(pages, hkv, page):
    """Strides that address nothing (3 for a dimension of one) are not looked at."""
    d = 64
    kc, vc = (randn(pages, hkv, page, d, seed=s).to(DEV) for s in (1, 2))
    odd = [3 if n == 1 else s for n, s in zip(kc.shape, kc.stride())]
    kv = [t.as_strided(t.shape, odd) for t in (kc, vc)]
    table, ctx = torch.arange(pages, dtype=torch.int32, device=DEV)[None], [pages * page - 2]
    q = randn(2, 4, d, seed=3).to(DEV)
    for k, v in (kv, (kv[0], vc)):
        out = block.awq_attn_tree(q, k, v, table, i32(ctx), cumulative([2]), 2)
        ref.check(out, *ref.tree(q, kc, vc, table, ctx, [2], None))
    freq, _ = block.rope_frequencies(d, device=DEV)
    new = randn(1, hkv, d, seed=4).to(DEV)
    block.awq_rope(None, i32([0]), freq, k=new, v=new, k_cache=kv[0], v_cache=kv[1],
                   slots=torch.tensor([pages * page - 1], device=DEV))
    assert torch.equal(vc[-1, :, -1], new[0]) and torch.equal(kc[-1, :, -1], new[0])


# ------------------------------------------------------ what infinities and NaN cost, and do

def milliseconds(call):
    call()
    times = []
    for _ in range(3):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        call()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
    return min(times)


# What a NaN costs: the products of a wavefront's tiles once more, with loads that nothing hides (a
# few times the call's 0.2 ms), and for a tile or step that holds it and is not seen whole by
# every row, key by key, at most 64 keys (two rows of loads each, 5 us if nothing overlaps, 0.3 ms;
# with 4096 wavefronts of which 2048 run at once twice that). Whole rows key by key took
# 114 ms with one NaN in the first value.

@pytest.mark.parametrize("where", ["first value", "first key", "every value", "every key", "last value", "value 2000"])
def test_a_visible_nan_does_not_slow_a_prompt_down(where):
    n, hq, hkv, d = 4096, 32, 8, 128
    q, k, v = randn(n, hq + 2 * hkv, d, seed=1).to(DEV).split([hq, hkv, hkv], 1)
    cu = cumulative([n])
    target = k if "key" in where else v
    first, last = {"first": (0, 1), "every": (0, n), "last": (n - 1, n), "value": (2000, 2001)}[where.split()[0]]
    target[first:last, 0, 7] = float("nan")
    assert milliseconds(lambda: block.awq_attn_prompt(q, k, v, cu)) < 2.0
    nan = torch.isnan(block.awq_attn_prompt(q, k, v, cu))
    hit = torch.zeros_like(nan)
    hit[first:, :4, :] = "key" in where
    hit[first:, :4, 7] = True
    assert torch.equal(nan, hit)


@pytest.mark.parametrize("drafts", [1, 8, 64])
def test_a_visible_nan_does_not_slow_drafts_down(drafts):
    ctx, hq, hkv, d, page = [20000], 32, 8, 128, 16
    q, kc, vc, table = tree_inputs(ctx, [drafts], hq, hkv, d, page, F16, seed=drafts)
    n, cu = i32(ctx), cumulative([drafts])
    for pos in (0, 9999, 20000):
        vc[at(table, 0, pos, page) + (7,)] = float("nan")
    assert milliseconds(lambda: block.awq_attn_tree(q, kc, vc, table, n, cu, drafts)) < 2.0
    nan = torch.isnan(block.awq_attn_tree(q, kc, vc, table, n, cu, drafts))
    assert bool(nan[..., 7].all()) and int(nan.sum()) == drafts * hq


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [128, 64, 40])
def test_prompt_rows_before_a_bad_token(dtype, bad, d):
    """One token's value holds an infinity or NaN in a channel, at every place of a tile: the rows
    before it are right everywhere, the rows from it on in the other channels."""
    lengths, hq, hkv = [40, 333, 33], 4, 2
    qkv = randn(sum(lengths), hq + 2 * hkv, d, seed=d, dtype=dtype, gain=1.5)
    want, bound = ref.prompt(*qkv.split([hq, hkv, hkv], 1), lengths)
    for token in (0, 31, 32, 50, 63, 64, 100, 127, 128, 149, 250, 319, 332):
        x = qkv.clone()
        x[40 + token, hq + hkv:, 3] = bad
        out = block.awq_attn_prompt(*x.to(DEV).split([hq, hkv, hkv], 1), cumulative(lengths))
        hit = torch.zeros(want.shape, dtype=torch.bool)
        hit[40 + token:373, :, 3] = True
        assert not bool(torch.isfinite(out.cpu()[hit]).any()), token
        assert int(torch.isnan(out).sum()) == (int(hit.sum()) if bad != bad else 0), token
        ref.check(torch.where(hit, 0.0, out.cpu()), torch.where(hit, 0.0, want), bound, f"token {token}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
@pytest.mark.parametrize("ctx", [[64, 300], [3000, 90]])
def test_drafts_of_which_some_are_bad(dtype, bad, ctx):
    """64 drafted tokens, some of them bad in one channel: rows that do not see one are right, the
    others in the other channels, wherever the new tokens start in a step."""
    drafts, hq, hkv, d, page = [64, 61], 4, 2, 72, 16
    for shift in (0, 1, 17, 31, 40):
        at_ctx = [c + shift for c in ctx]
        q, kc, vc, table = tree_inputs(at_ctx, drafts, hq, hkv, d, page, dtype, seed=shift)
        masks = tree_masks(drafts, shift)
        want, bound = ref.tree(q, kc, vc, table, at_ctx, drafts, masks)
        hit = torch.zeros(want.shape, dtype=torch.bool)
        for b in range(2):
            for j in (0, 3, 33, 60):
                vc[at(table, b, at_ctx[b] + j, page) + (5,)] = bad
                for t in range(drafts[b]):
                    hit[b * 64 + t, :, 5] |= bool(masks[b * 64 + t] >> j & 1)
        out = block.awq_attn_tree(q, kc, vc, table, i32(at_ctx), cumulative(drafts), 64, mask=words(masks)).cpu()
        assert not bool(torch.isfinite(out[hit]).any())
        ref.check(torch.where(hit, 0.0, out), torch.where(hit, 0.0, want), bound, f"shift {shift}")


# ------------------------------------------------------------- values of any size in bfloat16

def wide_values(g, n, d, gain):
    v = torch.randn(n, 1, d, generator=g) * gain
    return v.clamp(-3.38e38, 3.38e38).to(BF16)   # (the type's largest is 3.39e38)


@pytest.mark.parametrize("gain", [1e-25, 1e25, 1e31, 1e37, 3e38])
def test_prompt_values_of_any_size(gain):
    """Rows whose maximum moves from key to key; the bound is relative to the values."""
    g = torch.Generator().manual_seed(13)
    for n, spread in ((400, 8.0), (1500, 0.0)):   # (spread 0: every key weighs the same)
        q = (torch.randn(n, 1, 64, generator=g) * 6).to(BF16)
        k = (torch.randn(n, 1, 64, generator=g) * torch.linspace(0.1 * spread, spread, n)[:, None, None]).to(BF16)
        v = wide_values(g, n, 64, gain)
        v[:, :, 5] = 3.38e38 if gain > 1e38 else v[:, :, 5]
        out = block.awq_attn_prompt(q.to(DEV), k.to(DEV), v.to(DEV), cumulative([n]))
        assert bool(torch.isfinite(out).all())
        ref.check(out, *ref.prompt(q, k, v, [n]))


@pytest.mark.parametrize("gain", [1e-25, 1e25, 1e31, 1e37, 3e38])
@pytest.mark.parametrize("ctx,drafts,hq", [([50], [1], 4), ([50], [40], 4), ([5000], [2], 4), ([5000], [20], 4)])
def test_tree_values_of_any_size(gain, ctx, drafts, hq):
    q, kc, vc, table = tree_inputs(ctx, drafts, hq, 1, 128, 16, BF16, seed=5)
    g = torch.Generator().manual_seed(6)
    vc[:] = wide_values(g, vc.shape[0] * 16, 128, gain).view(-1, 1, 16, 128).to(DEV)
    kc *= 3
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), max(drafts))
    assert bool(torch.isfinite(out).all())
    ref.check(out, *ref.tree(q, kc, vc, table, ctx, drafts, None))


# ---------------------------------------------------------- the sum of what is multiplied

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("ctx,drafts,hq", [([300], [1], 4), ([300], [9], 4), ([6000], [1], 4)])
def test_equal_values_come_out_as_they_are(dtype, ctx, drafts, hq):
    """Every value row is the same, and beside a largest score in every 16 positions all are such
    that the probabilities round up by most of half a step: the weights' sum has to be that of
    the rounded ones."""
    y = -torch.arange(1, 800, dtype=torch.float64).div(1024).to(dtype).double().unique()
    p = torch.exp(y)
    up = p.to(dtype).double() / p - 1
    score = float(y[up.argmax()])
    assert float(up.max()) > 0.8 * ref.U[dtype]
    q, kc, vc, table = tree_inputs(ctx, drafts, hq, 1, 128, 16, dtype, seed=1)
    q[:], kc[:] = 0, 0
    q[..., 0], kc[..., 0] = 1, score
    kc[:, :, 0, 0] = 0
    value = randn(128, seed=2, dtype=dtype).to(DEV)
    vc[:] = value
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), max(drafts), scale=1.0)
    assert torch.equal(out, value.expand_as(out))


# ------------------------------------------- block tables much wider than the contexts in them

@pytest.mark.parametrize("ctx,drafts", [([517], [1]), ([517, 0, 90, 2000], [3, 1, 12, 30])])
def test_a_table_for_the_longest_context(ctx, drafts):
    """As a captured decode step has one: 32768 positions, the entries past a sequence's pages
    anything; the splits past its end leave nothing behind."""
    q, kc, vc, narrow = tree_inputs(ctx, drafts, 8, 2, 128, 16, F16, seed=8)
    table = torch.full((len(ctx), 2048), -7, dtype=torch.int32, device=DEV)
    table[:, :narrow.shape[1]] = narrow
    table[:, 1000:] = 1 << 30
    assert splits(q, kc, table, max(drafts)) > splits(q, kc, narrow, max(drafts))
    masks = tree_masks(drafts, 9)
    need = block.awq_attn_tree_workspace_bytes(sum(drafts), len(ctx), 2048, 16, max(drafts), 8, 2, 128)
    ws = torch.full((need // 4,), float("nan"), device=DEV).view(torch.uint8)
    out = block.awq_attn_tree(q, kc, vc, table, i32(ctx), cumulative(drafts), max(drafts), mask=words(masks), ws=ws)
    ref.check(out, *ref.tree(q, kc, vc, narrow, ctx, drafts, masks))
