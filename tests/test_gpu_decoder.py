"""The operators together, as examples/decoder_blocks.py uses them: a tree of drafted tokens in
one pass against the same tokens decoded one by one."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("bit_weight_only_w4a16_amd.block")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [(37, 5, 64), (1, 130, 16)])
def test_tree_pass_matches_token_by_token_decoding(lengths):
    import decoder_blocks
    diff, top = decoder_blocks.run(lengths, seed=sum(lengths))
    # two layers of binary16 activations, each rounded a handful of times in another order
    # (products of 1 and of several rows differ by the weights' rounding): 2e-3 of the
    # largest value per product, the products' documented accuracy, over ten products in a row
    assert diff <= 10 * 2e-3 * top
    assert top > 0.5


def test_quant_linear_with_a_tail():
    """QuantLinear hands a tail to the fused product."""
    from bit_weight_only_w4a16_amd import awq, block
    g = torch.Generator().manual_seed(3)
    w = (torch.randn(264, 256, generator=g) * 0.05).half().cuda()
    layer = awq.QuantLinear.from_weight(w, torch.randn(32, 256, generator=g).half().cuda())
    x, r = torch.randn(5, 256, generator=g).half().cuda(), torch.randn(5, 264, generator=g).half().cuda()
    want = block.awq_gemm_fused(x, layer.inv_s_c, layer.packed, 264, 256, act="silu", mul=r, residual=r)
    assert torch.equal(layer(x, act="silu", mul=r, residual=r), want)
    assert torch.equal(layer(x), awq.awq_gemm(x, layer.inv_s_c, layer.packed, 264, 256))
    assert torch.equal(layer(x, bias=r[0]), block.awq_gemm_fused(x, layer.inv_s_c, layer.packed, 264, 256, bias=r[0]))
