"""GPU tests of bf16 prompts of linear attention: the precision that the header states."""
from __future__ import annotations

import pytest
import torch

from test_gpu_linattn import Case

pytestmark = pytest.mark.gpu


def relative(got, want):
    return float((got.detach().cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_bf16_prompt_precision_is_the_stated_one(cuda_lib, dk, dv):
    """What the header says of bf16 prompts: the products with q are of bf16 operands.  Scores and state are rounded
    by at most 2^-8 each, a term is in one of the two sums, and out is rounded once more: of errors that are independent
    of one another, sqrt(2) * 2^-8 of the outputs' norm."""
    c = Case(2, 1, 2, dk, dv, "bf16", counts=[1000, 300], gain=True, seed=31, decay=0.01)
    d = c.prefill(cuda_lib)
    out, _, state, _ = c.expect(True)
    assert relative(d["out"], out) < 2 ** 0.5 * 2.0 ** -8
    slots = c.slot.long()
    assert relative(d["state"].cpu()[slots], state[slots]) < 2.0 ** -15
