"""examples/expert_layer.py: the layer learns, and its fp8 form answers as its bf16 form does."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,inner,experts", [(300, 256, 128, 8), (513, 200, 333, 5)])
def test_expert_layer_trains_and_serves(gpu_available, tokens, hidden, inner, experts):
    import expert_layer
    losses, errors = expert_layer.run(tokens, hidden, inner, experts, out=64, steps=40)
    assert all(math.isfinite(v) for v in losses) and losses[-1] < 0.5 * losses[0]
    # Each product has two quantised operands, a value of which is off by at most 2^-4 of itself
    # independently of the others; three products in a row: sqrt(6) * 2^-4 of the outputs' norm.
    assert all(e < 6 ** 0.5 / 16 for e in errors), errors
