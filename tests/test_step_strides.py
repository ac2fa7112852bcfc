"""Rows that are one (stride 0): which calls take them, on the host (no rows, so nothing is launched)."""
import pytest

from block_quantized_weight_q4_gb300 import binding
from block_quantized_weight_q4_gb300.build import build

OK, SHAPE = 0, 3
P = 1 << 20


@pytest.mark.parametrize("stride,ns,want", [(0, 100, OK), (100, 0, OK), (0, 0, OK), (1, 100, SHAPE), (99, 0, SHAPE), (0, 99, SHAPE), (-1, 100, SHAPE),
                                            (100, -100, SHAPE)])
def test_sample(stride, ns, want):
    build()
    assert binding.load_library().qmv_sample(0, 100, P, stride, P, ns, None, None, None, None, P, None) == want
