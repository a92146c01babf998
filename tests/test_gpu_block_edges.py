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
