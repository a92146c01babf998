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
