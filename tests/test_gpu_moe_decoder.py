"""The feed-forward operators together, as examples/moe_decoder.py uses them."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("bit_weight_only_w4a16_amd.moe")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [(37, 5, 64), (1, 130, 16)])
def test_a_token_decoded_alone_is_the_prompts(lengths):
    import moe_decoder
    eight, four, want, got = moe_decoder.run(lengths, seed=sum(lengths))
    assert eight.shape == four.shape == (sum(lengths), 512)
    assert bool(torch.isfinite(eight).all()) and bool(torch.isfinite(four).all())
    # the same formats in another order of sums and roundings: 2e-3 of the largest value for each
    # product (the products' documented accuracy), over ten products in a row
    assert float((want.float() - got.float()).abs().max()) <= 10 * 2e-3 * float(want.float().abs().max())
