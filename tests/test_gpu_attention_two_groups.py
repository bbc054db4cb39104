"""More rows than one tile of the tensor-core kernel (two groups of softmax warps, each with rows of its own), and heads of 129 to 256
channels: values that are not finite, and waits that run out."""
from __future__ import annotations

import pytest
import torch

import attn_reference as ref
from test_gpu_attention import BF, call, check, make

pytestmark = pytest.mark.gpu
SHAPES = [  # drafts, query heads a kv head, head size
    (9, 16, 128), (17, 8, 64), (70, 2, 128), (3, 64, 64), (9, 3, 192), (9, 3, 256), (9, 3, 128)]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens", [[5], [100, 126], [3, 700]], ids=str)
@pytest.mark.parametrize("T,G,d", SHAPES)
def test_values_that_are_not_finite_stay_where_they_are_seen(cuda_lib, T, G, d, lens, bad):
    """One draft's v (or k) of each sequence reaches its descendants and nobody else."""
    n, at = len(lens), T // 2
    for which in "kv":
        x = make(lens, [T] * n, T, 1, G, d, 16, BF, tree=True, seed=T)
        rows = [x["table"][int(s)] for s in x["slots"]]
        for L, row in zip(lens, rows):
            x[which][int(row[(L + at) // 16]), (L + at) % 16, 0, 7] = bad
        out, err = call(cuda_lib, x)
        assert err == [0] * n
        for s, (L, row) in enumerate(zip(lens, rows)):
            seen = ref.ancestors(x["parents"][s])
            K, V = (ref.gather(x[c], row, L + T).nan_to_num(0, 0, 0) for c in "kv")
            want, size, top = ref.attention(x["q"][s].double(), K, V, L, x["parents"][s], d ** -0.5)
            bound = ref.attention_bound(BF, want, size, top, L + T, d)
            right = (out[s].double() - want).abs() <= bound
            keep = torch.arange(d) != 7
            for t in range(T):
                if at not in seen[t]:
                    assert bool(right[t].all()), (s, t)
                elif which == "v":
                    assert bool(right[t][:, keep].all()) and bool((~torch.isfinite(out[s, t, :, 7])).all())
                    assert bad != bad or bool((out[s, t, :, 7] == bad).all())


def inputs(kind):
    if kind == "cut":
        return make([9000, 3000], [17, 17], 17, 1, 16, 128, 16, BF, tree=True, seed=1)
    return make([200] * 20, [9] * 20, 9, 2, 16, 64, 16, BF, seed=3, pad=(3, 19))


@pytest.mark.parametrize("kind", ["cut", "many"])
def test_waits_give_up_at_once(cuda_lib, kind):
    x = inputs(kind)
    out, err = call(cuda_lib, x, wait_polls=-1)
    assert err == [8 if s >= 0 else 0 for s in x["slots"].tolist()]
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("polls", [1, 2, 4])
@pytest.mark.parametrize("kind", ["cut", "many"])
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
