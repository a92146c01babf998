"""Sizes of the feed-forward operators' workspaces at and past their limits, without a GPU."""
import os

import pytest

pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
moe = pytest.importorskip("bit_weight_only_w4a16_amd.moe")

pytestmark = pytest.mark.skipif(not os.path.exists(awq.LIB_PATH), reason="library not built")


@pytest.mark.parametrize("tokens,hidden,ffn,k", [
    (4, 8, 384, 2), (4, 16, 384, 2), (4, 31, 384, 2), (4, 100, 384, 2), (4, 320, 384, 2), (4, 256, 100, 2), (4, 256, 8, 2),
    (4, 1 << 17, 1 << 14, 2), (4, 1 << 23, 128, 2), (4, 128, 1 << 23, 2), (0, 256, 384, 2), (-1, 256, 384, 2),
    (65, 256, 384, 2), (4, 0, 384, 2), (4, 256, -128, 2), (4, 256, 384, 0), (4, 256, 384, 33),
])
def test_moe_workspace_of_refused_sizes_is_0(tokens, hidden, ffn, k):
    assert moe.awq_moe_workspace_bytes(tokens, hidden, ffn, k) == 0


@pytest.mark.parametrize("tokens,hidden,ffn,k", [
    (1, 128, 128, 1), (64, 128, 128, 32), (1, 8192, 640, 2), (64, 1 << 22, 128, 1), (64, 128, 1 << 22, 32),
    (64, 1 << 15, (1 << 16) - 128, 32),
])
def test_moe_workspace_holds_the_second_products_operand(tokens, hidden, ffn, k):
    assert moe.awq_moe_workspace_bytes(tokens, hidden, ffn, k) >= 2 * tokens * k * ffn
