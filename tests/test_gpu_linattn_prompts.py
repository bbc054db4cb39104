"""GPU tests of bf16 prompts of linear attention: the precision that the header states, also along long prompts."""
from __future__ import annotations

import pytest
import torch

from layer_reference import assert_within, linattn
from test_gpu_linattn import Case

pytestmark = pytest.mark.gpu


def relative(got, want):
    return float((got.detach().cpu().double() - want).norm() / want.norm())


def copies(c, n):
    """The one prompt of `c` n times over, in as many sequences of one call (each from its own copy of the state)."""
    big = Case(n, c.nq, c.nh, c.dk, c.dv, "bf16" if c.dtype == torch.bfloat16 else "f32", counts=c.counts * n, seed=1)
    x = c.tok["x"].repeat(n, 1)
    for t in "qkv":
        big.tok[t] = x.as_strided((x.shape[0], *c.tok[t].shape[1:]), c.tok[t].stride(), c.tok[t].storage_offset())
    big.tok.update(x=x, g=c.tok["g"].repeat(n, 1), b=c.tok["b"].repeat(n, 1) if c.tok["b"] is not None else None)
    big.state_wide[big.slot.long()] = c.state_wide[int(c.slot[0])].clone()
    return big


def workspace(cv, c, d):
    return cv.linattn_workspace(d["q"], d["k"], d["v"], d["g"], d["state"], d["out"], d["cu"], max_seqlen=c.T)


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


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("length,n,cut", [(2048, 1, True), (2048, 160, False), (8192, 1, True), (8192, 160, False),
                                          (32768, 1, True)])
def test_state_keeps_its_bits_along_a_prompt(cuda_lib, length, n, cut, positive):
    """The error of the state that a long prompt leaves, with decays near one, so that every chunk's roundings stay in
    it.  Its terms carry 17 bits (2^-17 each); the sums are fp32.  Losing the keys' low part would
    leave 1.7e-3, a state rounded to bf16 between chunks 4e-3."""
    c = Case(1, 1, 1, 64, 64, "bf16", counts=[length], seed=length, decay=0.0005)
    if positive:
        c.tok["x"].abs_()
    _, want, _, _ = linattn(c.state[int(c.slot[0])], None, c.tok["k"], c.tok["v"], c.tok["g"])
    big = copies(c, n) if n > 1 else c
    d = big.device()
    assert (workspace(cuda_lib, big, d) > 0) == cut
    big.prefill(cuda_lib, d)
    got = d["state"].cpu()[big.slot.long()]
    err = [relative(x, want) for x in got]
    print(f"length {length} n {n} positive {positive}: {max(err):.2e}")
    assert max(err) < 2.0 ** -15


def timed(run, passes=5):
    """The shortest of a few passes, in us."""
    run()
    best = float("inf")
    for _ in range(passes):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        run()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("where", [(3,), (0, 9, 64, 127), tuple(range(128))])
def test_an_infinity_in_every_chunk_costs_little(cuda_lib, where):
    """A prompt whose v overflowed here and there takes about as long as any other: each of the 16 groups of 8 columns
    is 1/16 of A V again, a product at a time, which is no more than the whole chunk; 20 times covers all of them."""
    c = Case(1, 1, 1, 128, 128, "bf16", counts=[16 * 128], seed=41)
    d = c.device()
    run = lambda: cuda_lib.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["state"], d["out"], d["cu"],  # noqa: E731
                                           max_seqlen=c.T, cache_idx=d["slot"])
    clean = timed(run)
    d["v"][5::128, 0, list(where)] = float("inf")
    bad = timed(run)
    print(f"columns {len(where)}: {clean:.1f} us, with an infinity in every chunk {bad:.1f}")
    assert bad < 20 * clean


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (40, 96)])
@pytest.mark.parametrize("decay", [0.1, 3.0])
@pytest.mark.parametrize("skip", [False, True])
def test_nonfinite_values_spoil_their_columns_alone(cuda_lib, dk, dv, decay, skip):
    """NaN and infinities in v, several a chunk and in some chunks only: every other column of every output is as
    without them, before and after, and so are the spoiled columns' outputs up to the first bad token."""
    c = Case(3, 1, 2, dk, dv, "bf16", counts=[700, 130, 260], seed=42, gain=True, skip=skip, decay=decay)
    clean = Case(3, 1, 2, dk, dv, "bf16", counts=[700, 130, 260], seed=42, gain=True, skip=skip, decay=decay)
    v = c.tok["v"]
    bad = [(130, 0, 3, float("inf")), (131, 0, 3, float("nan")), (200, 1, dv - 1, float("-inf")), (255, 0, 17, float("nan")),
           (640, 1, 8, float("inf")), (700 + 127, 0, 0, float("inf")), (830 + 3, 1, 5, float("nan"))]
    for t, h, col, x in bad:
        v[t, h, col] = x
    d = c.prefill(cuda_lib)
    out, lim, state, slim = clean.expect(True, chunked=True)
    ok = torch.ones_like(out, dtype=torch.bool)
    fine = torch.ones_like(state, dtype=torch.bool)
    for t, h, col, _ in bad:
        s = 0 if t < 700 else 1 if t < 830 else 2
        ok[t:c.cu[s + 1], h, col] = False
        fine[int(c.slot[s]), h, :, col] = False
    assert not torch.isfinite(torch.stack([d["out"][t, h, col] for t, h, col, _ in bad])).any()
    got, left = d["out"].cpu().double(), d["state"].cpu().double()
    assert ((got - out).abs()[ok] <= lim.expand_as(out)[ok]).all()
    assert ((left - state).abs()[fine] <= slim.expand_as(state)[fine]).all()


@pytest.mark.parametrize("counts,nh,dk,dv", [([300, 140], 2, 64, 64), ([3000, 200], 1, 64, 128), ([500], 2, 40, 96),
                                             ([1200, 129], 1, 128, 128)])
@pytest.mark.parametrize("where", ["k", "v", "both"])
@pytest.mark.parametrize("gain", [False, True])
def test_the_state_holds_the_infinities_of_the_definition(cuda_lib, counts, nh, dk, dv, where, gain):
    """Infinities and NaN in k and v leave those infinities and NaN in the state that the recurrence does (inf + finite
    stays inf, inf - inf is NaN), in the pieces of cut prompts and in whole ones, and all else as it is."""
    c = Case(len(counts), 1, nh, dk, dv, "bf16", counts=counts, seed=43, gain=gain, decay=0.02)
    d = c.device()
    assert (workspace(cuda_lib, c, d) > 0) == (counts[0] >= 1000)
    inf = float("inf")
    if where != "v":
        c.tok["k"][130, 0, 3], c.tok["k"][131, 0, 5], c.tok["k"][250, 0, 5] = inf, -inf, inf
        c.tok["k"][counts[0] - 1, 0, 8] = float("nan")
    if where != "k":
        c.tok["v"][5, 0, 3], c.tok["v"][200, 0, 9], c.tok["v"][201, nh - 1, dv - 1] = inf, -inf, -inf
        c.tok["v"][290, 0, 0], c.tok["v"][290, 0, dv - 8] = float("nan"), inf
    d = c.prefill(cuda_lib)
    _, _, state, slim = c.expect(True, chunked=True)
    assert torch.isinf(state).any() and d["err"].tolist() == [0] * len(counts)
    assert_within(d["state"], state, slim, "state")


def test_infinite_gains_and_initial_states(cuda_lib):
    c = Case(2, 1, 2, 64, 64, "bf16", counts=[300, 150], seed=44, gain=True, decay=0.02)
    c.tok["b"][140, 0], c.tok["b"][20, 1] = float("inf"), float("nan")
    c.state[int(c.slot[1]), 0, 7, 9], c.state[int(c.slot[1]), 1, 3, 4] = float("-inf"), float("nan")
    d = c.prefill(cuda_lib)
    _, _, state, slim = c.expect(True, chunked=True)
    assert_within(d["state"], state, slim, "state")


def mix_decays(c, pattern, drops=True):
    """Per chunk of 128 tokens and head: w slow decays, s strong ones (0.5 to 2 a token: 2^-92 to 2^-370 a chunk), d
    strong ones with tokens that drop the state; sequence and head shift the pattern."""
    for s in range(c.n):
        for h in range(c.nh):
            for i, lo in enumerate(range(c.cu[s], c.cu[s + 1], 128)):
                hi, kind = min(lo + 128, c.cu[s + 1]), pattern[(i + s + 2 * h) % len(pattern)]
                r = torch.rand(hi - lo, generator=c.rng)
                c.tok["g"][lo:hi, h] = -0.02 * r if kind == "w" else -0.5 - 1.5 * r
                if kind == "d" and drops:
                    c.tok["g"][lo + 7:hi:23, h] = float("-inf")
                    c.tok["g"][lo + 40:lo + 44, h][:max(0, hi - lo - 40)] = torch.finfo(torch.float32).min


@pytest.mark.parametrize("pattern,n,nh,dk,dv,skip,gain", [
    ("wwsds", 20, 8, 64, 64, False, False), ("sd", 20, 8, 128, 128, True, True), ("wsws", 20, 8, 128, 128, False, False)] + [
    (pattern, n, nh, dk, dv, skip, gain) for pattern in ("ws", "wwsds", "sd", "wdws")
    for n, nh, dk, dv, skip, gain in ((3, 2, 64, 128, True, False), (2, 1, 128, 64, False, True))])
def test_weak_and_strong_chunks_follow_one_another(cuda_lib, pattern, n, nh, dk, dv, skip, gain):
    """The kernel's two forms of a chunk in every order, across a block's units (more units than SMs) and within cut prompts."""
    counts = [430 - 13 * s for s in range(n)] if n > 3 else [1500, 900, 641][:n]
    c = Case(n, 1, nh, dk, dv, "bf16", counts=counts, seed=61, skip=skip, gain=gain)
    mix_decays(c, pattern)
    d = c.prefill(cuda_lib)
    c.check(d, True, chunked=True)
    again = c.prefill(cuda_lib)
    assert torch.equal(d["out"], again["out"]) and torch.equal(d["state"], again["state"])


@pytest.mark.parametrize("scale", [5e-5, 0.0, -1e-3])
def test_skip_beside_a_small_scale(cuda_lib, scale):
    """The skip weight enters the scores divided by scale, unless that is too small: then as strong chunks do it."""
    c = Case(2, 1, 2, 64, 64, "bf16", counts=[300, 140], seed=62, skip=True, gain=True)
    c.scale = scale
    c.check(c.prefill(cuda_lib), True, chunked=True)


def test_dropped_states_many_to_a_block(cuda_lib):
    """Half of a block of 32 tokens drops the state, the other half decays slowly."""
    c = Case(1, 1, 2, 64, 64, "bf16", counts=[256], seed=63)
    c.tok["g"].mul_(0.01)
    for lo in range(0, 256, 32):
        c.tok["g"][lo:lo + 16] = float("-inf")
    c.check(c.prefill(cuda_lib), True, chunked=True)


@pytest.mark.parametrize("n,nh,longest,cut", [(70, 4, 300, False), (66, 1, 2600, True), (65, 1, 260, False)])
def test_more_sequences_than_are_sorted(cuda_lib, n, nh, longest, cut):
    counts = [longest if s % 33 == 5 else (s * 37) % 250 for s in range(n)]
    c = Case(n, 1, nh, 64, 64, "bf16", counts=counts, seed=64, pad_seqs=(3, n - 1), no_init=range(0, n, 4), decay=0.01)
    d = c.device()
    assert (workspace(cuda_lib, c, d) > 0) == cut
    c.check(c.prefill(cuda_lib, d), True, chunked=True)


def test_more_recurrent_sequences_than_are_counted(cuda_lib):
    counts = [1800 if s == 7 else (s * 41) % 120 for s in range(40)]
    c = Case(40, 1, 1, 64, 64, "f32", counts=counts, seed=65, pad_seqs=(9,), no_init=(0, 7), decay=0.01)
    d = c.device()
    assert workspace(cuda_lib, c, d) > 0
    c.check(c.prefill(cuda_lib, d), True)


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("counts,nh", [([1500], 1), ([1500, 40], 60)])
def test_an_infinity_outlives_small_decays_but_no_drop(cuda_lib, counts, nh, dropped):
    """An infinity in the state stays one under decays that multiply to far less than fp32 holds, within a chunk, over a
    whole prompt and over the pieces of a cut one; a token that drops the state makes it a NaN (0 * inf)."""
    c = Case(len(counts), 1, nh, 64, 64, "bf16", counts=counts, seed=66)
    d = c.device()
    assert (workspace(cuda_lib, c, d) > 0) == (nh == 1)
    c.tok["v"][3, 0, 5] = float("inf")
    c.tok["g"][200:700, 0] = -2.0
    if dropped:
        c.tok["g"][450, 0] = float("-inf")
    d = c.prefill(cuda_lib)
    _, _, state, slim = c.expect(True, chunked=True)
    assert bool(torch.isinf(state).any()) != dropped
    assert_within(d["state"], state, slim, "state")
