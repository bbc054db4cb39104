"""The bounded waits of the attention kernel, given up at once or after a few polls (no fault: an ordinary wait runs out).  The
call returns and flags every sequence it did not finish; all others, and the next call, are right."""
from __future__ import annotations

import pytest
import torch

from test_gpu_attention import BF, call, check, make

pytestmark = pytest.mark.gpu


def inputs(kind):
    if kind == "cut":
        return make([9000, 3000], [4, 4], 4, 1, 4, 128, 16, BF, tree=True, seed=1)
    if kind == "wide":
        return make([300, 5, 700], [9, 9, 9], 9, 2, 2, 256, 32, BF, tree=True, seed=2, pad=(1,))
    return make([200] * 60, [3] * 60, 3, 4, 2, 64, 16, BF, seed=3, pad=(3, 59))


@pytest.mark.parametrize("kind", ["cut", "wide", "many"])
def test_waits_give_up_at_once(cuda_lib, kind):
    x = inputs(kind)
    out, err = call(cuda_lib, x, wait_polls=-1)
    assert err == [8 if s >= 0 else 0 for s in x["slots"].tolist()]
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("polls", [1, 2, 4])
@pytest.mark.parametrize("kind", ["cut", "wide", "many"])
def test_short_waits_leave_the_others_right(cuda_lib, kind, polls):
    x = inputs(kind)
    out, err = call(cuda_lib, x, wait_polls=polls)
    assert set(err) <= {0, 8}
    for s, e in enumerate(err):
        if e:
            x["slots"][s] = -1
            out[s] = 7
    check(x, out, err)
    x = inputs(kind)
    check(x, *call(cuda_lib, x))
