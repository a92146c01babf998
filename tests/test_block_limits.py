"""Limits of the decoder-block operators and values of their helpers, without a GPU."""
import ctypes
import math
import os

import pytest

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
block = pytest.importorskip("bit_weight_only_w4a16_amd.block")

import block_ctypes as c_abi  # noqa: E402

UNSUPPORTED = 2
P = 1 << 20   # an aligned stand-in address; never dereferenced, because validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(awq.LIB_PATH):
        pytest.skip("library not built")
    return c_abi.lib()


def test_tree_refuses_more_workgroups_than_a_launch_holds(lib):
    """64 tokens x 4096 heads of one group are 4096 row blocks; 2^29 positions in pages of one
    are 599187 splits: 2.5e9 workgroups (which also pass 32 bits)."""
    sizes = dict(tokens=64, seqs=1, table_width=1 << 29, page_size=1, max_q=64, q_heads=4096, kv_heads=1, head_dim=128)
    args = c_abi.AttnTreeArgs(q=P, k_cache=P, v_cache=P, out=P, block_table=P, ctx_lens=P, cu_q=P, ws=P,
                              ws_bytes=1 << 62, pages=100, q_token=4096 * 128, q_head=128, o_token=4096 * 128, o_head=128,
                              cache_page=128, cache_head=128, cache_slot=128, dtype=0, scale=0.1, **sizes)
    assert lib.awq_attn_tree(ctypes.byref(args), None) == UNSUPPORTED
    assert lib.awq_attn_tree_workspace_bytes(*sizes.values()) == 0
    # one head, the same table: as many splits, one row block
    sizes.update(q_heads=1)
    assert lib.awq_attn_tree_workspace_bytes(*sizes.values()) > 0


def test_stretched_frequencies_between_their_ends():
    """Each pair of the two blends, with their published bounds as the default: "bands" between 1
    and 4 turns over the original context, "yarn" between the pairs of 1 and 32 turns."""
    rot, base, factor, original = 128, 10000.0, 8.0, 4096
    freq = [base ** (-2 * i / rot) for i in range(rot // 2)]
    turns = [original * f / (2 * math.pi) for f in freq]
    bands = [min(max((t - 1.0) / 3.0, 0.0), 1.0) for t in turns]
    # the pairs of 32 turns and of 1: 128 ln(4096 / (2 pi n)) / (2 ln 10000) = 20.9, 45.03
    yarn = [1.0 - min(max((i - 20) / (46 - 20), 0.0), 1.0) for i in range(rot // 2)]
    for name, keep in (("bands", bands), ("yarn", yarn)):
        assert 0 < sum(0.01 < k < 0.99 for k in keep)
        got, _ = block.rope_frequencies(rot, base, scaling=name, factor=factor, original=original)
        want = [f * k + f / factor * (1 - k) for f, k in zip(freq, keep)]
        assert torch.allclose(got.double(), torch.tensor(want, dtype=torch.float64), rtol=2e-7, atol=0), name
    slow, _ = block.rope_frequencies(rot, base, scaling="yarn", factor=factor, original=original, high=4.0)
    assert not torch.equal(slow, got)
