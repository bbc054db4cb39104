"""The bounded waits of the prompt kernel of linear attention, given up at once or after a few polls (no fault: an
ordinary wait runs out).  The call returns and flags every sequence it did not finish; a cut prompt whose pieces' states
were not made is left untouched; all other sequences, and the next call, are right."""
from __future__ import annotations

import pytest
import torch

from layer_reference import assert_within
from test_gpu_linattn import SENT, Case
from test_gpu_linattn_prompts import workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,nh,dk,dv,pad", [
    ([3000, 2000], 1, 64, 64, ()),          # cut
    ([2500, 40, 1300], 1, 128, 128, (2,)),  # cut, beside one of a single piece and a padded one
    ([260] * 50, 8, 64, 128, (3, 49))])     # whole, several units a block
def test_waits_give_up_at_once(cuda_lib, counts, nh, dk, dv, pad):
    c = Case(len(counts), 1, nh, dk, dv, "bf16", counts=counts, seed=51, pad_seqs=pad, gain=True)
    d = c.device()
    cut = workspace(cuda_lib, c, d) > 0
    assert cut == (max(counts) > 1000)
    before = d["state"].clone()
    c.prefill(cuda_lib, d, wait_polls=-1)
    assert d["err"].tolist() == [0 if s in pad else 8 for s in range(len(counts))]
    for s, n in enumerate(counts):
        if s in pad or (cut and n > 1000):
            assert (d["out"][c.cu[s]:c.cu[s + 1]] == SENT).all()
            if s not in pad:
                assert torch.equal(d["state"][int(c.slot[s])], before[int(c.slot[s])])
    d["state"].copy_(before)
    c.prefill(cuda_lib, d)
    c.check(d, True, chunked=True)


def test_a_cut_prompt_without_err_is_left_untouched_too(cuda_lib):
    c = Case(1, 1, 2, 64, 64, "bf16", counts=[4000], seed=52)
    d = c.device()
    before = d["state"].clone()
    cuda_lib.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["state"], d["out"], d["cu"], max_seqlen=c.T, cache_idx=d["slot"],
                             wait_polls=-1)
    torch.cuda.synchronize()
    assert torch.equal(d["state"], before) and (d["out"] == SENT).all()


@pytest.mark.parametrize("polls", [1, 2, 4])
@pytest.mark.parametrize("counts,nh", [([260] * 50, 8), ([3000, 2000], 1)])
def test_short_waits_leave_the_others_right(cuda_lib, polls, counts, nh):
    c = Case(len(counts), 1, nh, 64, 64, "bf16", counts=counts, seed=53 + polls)
    d = c.prefill(cuda_lib, wait_polls=polls)
    err = d["err"].tolist()
    assert set(err) <= {0, 8}
    out, lim, state, slim = c.expect(True, chunked=True)
    for s, e in enumerate(err):
        if not e:
            at, sl = slice(c.cu[s], c.cu[s + 1]), int(c.slot[s])
            assert_within(d["out"][at], out[at], lim[at], f"out of {s}")
            assert_within(d["state"][sl], state[sl], slim[sl], f"state of {s}")
