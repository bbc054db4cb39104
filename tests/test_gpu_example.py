"""The example of a hybrid layer runs every operator together and checks itself."""
from __future__ import annotations

import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [0, 1])
def test_hybrid_layer(cuda_lib, seed):
    """Prompt, verify and commit against one long prompt: the projections' rows are bf16 and are made by matrix
    products of other shapes, so outputs (of size about 1, up to 5) may be a few bf16 places apart (one is 2^-6 at 4);
    the state is a sum of products of such rows."""
    import hybrid_layer
    d_out, d_state, d_conv = hybrid_layer.main(seed=seed)
    assert d_out < 0.125
    assert d_state < 0.02
    assert d_conv < 0.07
