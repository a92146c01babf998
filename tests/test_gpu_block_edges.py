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
