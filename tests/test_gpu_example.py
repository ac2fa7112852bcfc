"""examples/decode_layer.py: the products and the operators between them, for a prompt and token by token."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_prompt_and_token_by_token_agree():
    """The same tokens through the cache one by one (pages raised as they fill, other kernels) and in one prompt
    pass.  Both read levels within about a step of 1/127 of the page's largest value: a relative error of
    about 0.5% in keys and values, a few hundredths in logits of unit scale."""
    from block_quantized_weight_q4_gb300.build import build
    build()
    import decode_layer
    ids, picked, whole = decode_layer.run(layers=2, tokens=8)
    assert len(ids) == 8 and np.isfinite(picked).all()
    assert np.abs(picked - whole).max() < 0.2
