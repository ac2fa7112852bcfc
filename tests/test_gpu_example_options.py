"""examples/decode_layer.py with its options: it runs, and its log probabilities are numbers."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("how", [dict(experts=1), dict(experts=3, temperature=0.8, top_k=50, top_p=0.95), dict(temperature=1.2, top_p=0.5)])
def test_options(how):
    from block_quantized_weight_q4_gb300.build import build
    build()
    import decode_layer
    ids, picked, whole = decode_layer.run(layers=1, tokens=3, **how)
    assert len(ids) == 3 and np.isfinite(picked).all() and np.isfinite(whole).all() and (picked <= 0).all()
