"""GPU tests of linear attention with a decay for each head: the recurrent step (decoding, drafts with the
deferred commit) and packed prompts, against the fp64 recurrence."""
from __future__ import annotations

import math

import pytest
import torch

from layer_reference import assert_within, linattn, linattn_bounds

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


def make_tokens(rng, lead, nq, nh, dk, dv, dtype, gain, pad=0, decay=0.3):
    """CPU tokens as slices of one wide row (pad extra channels in front), like a conv output."""
    row = pad + 2 * nq * dk + nh * dv
    x = torch.randn(*lead, row, generator=rng).to(dtype)
    q = x[..., pad:pad + nq * dk].unflatten(-1, (nq, dk))
    k = x[..., pad + nq * dk:pad + 2 * nq * dk].unflatten(-1, (nq, dk))
    v = x[..., pad + 2 * nq * dk:].unflatten(-1, (nh, dv))
    g = -decay * torch.rand(*lead, nh, generator=rng) ** 3
    b = torch.rand(*lead, nh, generator=rng) if gain else None
    return dict(x=x, q=q, k=k, v=v, g=g, b=b)


def to_gpu(tok):
    """The same on the GPU, q, k and v still views of one buffer."""
    x = tok["x"].cuda()
    out = {n: x.as_strided(tok[n].shape, tok[n].stride(), tok[n].storage_offset()) for n in "qkv"}
    out["g"] = tok["g"].cuda()
    out["b"] = tok["b"].cuda() if tok["b"] is not None else None
    return out


def spans(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


SENT = -123.0  # representable in both types


class Case:
    """One call's inputs, its results from the library, and the fp64 reference."""

    def __init__(self, n, nq, nh, dk, dv, dtype="bf16", counts=None, T=None, gain=False, skip=False, seed=0, pad_seqs=(),
                 no_init=(), pad=0, decay=0.3, state_pad=0):
        self.rng = torch.Generator().manual_seed(seed)
        self.n, self.nq, self.nh, self.dk, self.dv, self.dtype = n, nq, nh, dk, dv, DT[dtype]
        self.counts = counts if counts is not None else [T] * n
        self.packed = counts is not None
        self.T = max(self.counts, default=0) if T is None else T
        self.cu = spans(self.counts) if self.packed else None
        self.lead = (self.cu[-1],) if self.packed else (n, T)
        self.tok = make_tokens(self.rng, self.lead, nq, nh, dk, dv, self.dtype, gain, pad, decay)
        self.skip = torch.randn(nh, generator=self.rng) if skip else None
        n_slots = n + 3
        wide = torch.randn(n_slots, nh, dk * dv + state_pad, generator=self.rng)
        self.state_wide = wide
        self.state = wide[:, :, :dk * dv].unflatten(-1, (dk, dv))
        self.slot = torch.randperm(n_slots, generator=self.rng)[:n].int()
        for s in pad_seqs:
            self.slot[s] = -1
        self.init = torch.ones(n, dtype=torch.int32)
        for s in no_init:
            self.init[s] = 0
        self.scale = 0.37
        self.prev = None

    def add_prev(self, T=None, counts=None, accept=None, gain=False):
        self.pcounts = counts if counts is not None else [T] * self.n
        self.pcu = spans(counts) if counts is not None else None
        lead = (self.pcu[-1],) if counts is not None else (self.n, T)
        self.prev = make_tokens(self.rng, lead, self.nq, self.nh, self.dk, self.dv, self.dtype, gain)
        self.pT = max(self.pcounts)
        self.accept = accept if accept is not None else [int(torch.randint(0, c + 1, (1,), generator=self.rng))
                                                         for c in self.pcounts]
        return self

    def rows(self, tok, cu, counts, s):
        lo, n = (cu[s], counts[s]) if cu is not None else (None, counts[s])
        pick = (lambda t: t[lo:lo + n]) if cu is not None else (lambda t: t[s, :n])
        return [pick(tok[x]) if tok[x] is not None else None for x in ("q", "k", "v", "g", "b")]

    def expect(self, update, chunked=False, skip_seqs=()):
        """(out, out bound, state, state bound), sentinels where nothing is written (bound 0)."""
        out = torch.full((*self.lead, self.nh, self.dv), SENT, dtype=torch.float64)
        lim = torch.zeros_like(out)
        state = self.state.double().clone()
        slim = torch.zeros_like(state)
        for s in range(self.n):
            sl = int(self.slot[s])
            if sl < 0 or s in skip_seqs:
                continue
            S0 = self.state[sl].double() if self.init[s] else torch.zeros_like(self.state[sl]).double()
            touched, n_all, S, M = not self.init[s], 0, S0, S0.abs()
            if self.prev is not None:
                a = self.accept[s]
                _, k, v, g, b = [x[:a] if x is not None else None for x in self.rows(self.prev, self.pcu, self.pcounts, s)]
                _, S, _, M = linattn(S0, None, k, v, g, b)
                n_all, touched = a, touched or a > 0
                state[sl], slim[sl] = (S, linattn_bounds(M, None, self.dk, a, self.dtype, chunked)) if touched else (
                    state[sl], slim[sl])
            q, k, v, g, b = self.rows(self.tok, self.cu, self.counts, s)
            o, S2, m, M2 = linattn(S, q, k, v, g, b, self.skip, self.scale)
            # the second run's magnitudes start from the first one's (M >= |S|)
            _, _, m, M2 = linattn(M, q.abs(), k.abs(), v.abs(), g, b.abs() if b is not None else None,
                                  self.skip.abs() if self.skip is not None else None, self.scale)
            n_all += self.counts[s]
            at = slice(self.cu[s], self.cu[s + 1]) if self.packed else s
            out[at] = o
            lim[at] = linattn_bounds(m, o, self.dk, n_all, self.dtype, chunked)
            if update and (self.counts[s] > 0 or not self.init[s]):
                state[sl], slim[sl] = S2, linattn_bounds(M2, None, self.dk, n_all, self.dtype, chunked)
        return out, lim, state, slim

    def device(self):
        d = to_gpu(self.tok)
        wide = self.state_wide.cuda()
        d["state"] = wide.as_strided(self.state.shape, self.state.stride())
        d["out"] = torch.full((*self.lead, self.nh, self.dv), SENT, dtype=self.dtype, device="cuda")
        d["slot"], d["init"] = self.slot.cuda(), self.init.cuda()
        d["skip"] = self.skip.cuda() if self.skip is not None else None
        d["cu"] = i32(self.cu).cuda() if self.packed else None
        d["err"] = torch.full((self.n,), -7, dtype=torch.int32, device="cuda")
        return d

    def prev_gpu(self, cv):
        p = to_gpu(self.prev)
        return cv.LinattnDrafts(p["k"], p["v"], p["g"], i32(self.accept).cuda(), gain=p["b"],
                                cu_draft=i32(self.pcu).cuda() if self.pcu is not None else None, T=self.pT)

    def step(self, cv, update, d=None, **kw):
        d = d or self.device()
        cv.linattn_step(d["q"], d["k"], d["v"], d["g"], d["state"], d["out"], gain=d["b"], skip=d["skip"],
                        scale=self.scale, update_state=update, prev=self.prev_gpu(cv) if self.prev is not None else None,
                        cache_idx=d["slot"], has_initial_state=d["init"], cu_draft=d["cu"], T=self.T, err=d["err"], **kw)
        torch.cuda.synchronize()
        return d

    def prefill(self, cv, d=None, max_seqlen=None, **kw):
        d = d or self.device()
        cv.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["state"], d["out"], d["cu"],
                           max_seqlen=self.T if max_seqlen is None else max_seqlen, gain=d["b"], skip=d["skip"],
                           scale=self.scale, cache_idx=d["slot"], has_initial_state=d["init"], err=d["err"], **kw)
        torch.cuda.synchronize()
        return d

    def check(self, d, update, chunked=False, err=None, skip_seqs=()):
        out, lim, state, slim = self.expect(update, chunked, skip_seqs)
        assert_within(d["out"], out, lim, "out")
        assert_within(d["state"], state, slim, "state")
        assert d["err"].tolist() == (err or [0] * self.n)


# ---------------------------------------------------------------------------------------------- step


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,T,nq,nh,dk,dv", [
    (1, 1, 1, 1, 128, 128), (3, 1, 2, 6, 128, 128), (2, 4, 1, 3, 64, 64), (5, 8, 2, 4, 64, 128), (2, 17, 1, 2, 128, 64),
    (3, 3, 1, 1, 1, 1), (2, 5, 2, 2, 7, 13), (1, 9, 1, 2, 256, 40), (2, 2, 1, 1, 200, 256), (70, 1, 4, 8, 128, 128),
    (90, 8, 2, 4, 128, 128), (1, 128, 1, 2, 32, 16), (40, 1, 8, 16, 64, 64)])
@pytest.mark.parametrize("update", [True, False])
def test_step_shapes(cuda_lib, n, T, nq, nh, dk, dv, dtype, update):
    c = Case(n, nq, nh, dk, dv, dtype, T=T, gain=n % 2 == 0, skip=T % 2 == 0, seed=n * 100 + T)
    c.check(c.step(cuda_lib, update), update)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,P,dk,dv", [(1, 1, 128, 128), (8, 8, 128, 128), (4, 3, 64, 96), (17, 17, 64, 32), (2, 128, 16, 24)])
@pytest.mark.parametrize("update", [True, False])
def test_step_commits_the_previous_drafts(cuda_lib, T, P, dk, dv, dtype, update):
    c = Case(7, 2, 4, dk, dv, dtype, T=T, gain=True, skip=True, seed=P, pad_seqs=(2,), no_init=(1, 4))
    c.add_prev(T=P, gain=True, accept=[0, 0, P, P, min(1, P), max(0, P - 1), P])
    c.check(c.step(cuda_lib, update), update)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_packed_drafts(cuda_lib, dtype):
    c = Case(6, 2, 4, 128, 64, dtype, counts=[3, 0, 17, 1, 8, 9], gain=True, seed=3, pad_seqs=(4,))
    c.add_prev(counts=[5, 2, 0, 17, 3, 1])
    c.check(c.step(cuda_lib, False), False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_commit_alone(cuda_lib, dtype):
    c = Case(5, 2, 4, 64, 64, dtype, T=0, seed=5, no_init=(3,)).add_prev(T=8, gain=True, accept=[0, 8, 1, 0, 5])
    d = c.device()
    cuda_lib.linattn_commit(c.prev_gpu(cuda_lib), d["state"], cache_idx=d["slot"], has_initial_state=d["init"],
                            err=d["err"])
    torch.cuda.synchronize()
    c.check(d, False)


def test_verify_then_commit_equals_decoding(cuda_lib):
    """Drafts verified together and committed as accepted leave the state that decoding them leaves."""
    c = Case(4, 2, 6, 128, 128, "f32", T=8, gain=True, skip=True, seed=11)
    verify = c.step(cuda_lib, False)
    assert torch.equal(verify["state"].cpu(), c.state)
    accept = [8, 1, 5, 3]
    cuda_lib.linattn_commit(cuda_lib.LinattnDrafts(verify["k"], verify["v"], verify["g"], i32(accept).cuda(),
                                                   gain=verify["b"]), verify["state"], cache_idx=verify["slot"])
    for s, a in enumerate(accept):
        q, k, v, g, b = c.rows(c.tok, None, c.counts, s)
        _, S, _, M = linattn(c.state[int(c.slot[s])], None, k[:a], v[:a], g[:a], b[:a])
        assert_within(verify["state"][int(c.slot[s])], S, linattn_bounds(M, None, 128, a, c.dtype, False), "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,state_pad,dk,dv", [(1, 0, 32, 32), (3, 1, 30, 36), (0, 3, 64, 64), (2, 0, 8, 9), (4, 4, 64, 64)])
def test_strides_and_alignments(cuda_lib, pad, state_pad, dk, dv, dtype):
    c = Case(3, 1, 2, dk, dv, dtype, T=3, gain=True, seed=pad, pad=pad, state_pad=state_pad)
    c.check(c.step(cuda_lib, True), True)
    p = Case(3, 1, 2, dk, dv, dtype, counts=[5, 70, 130], gain=True, seed=pad, pad=pad, state_pad=state_pad)
    p.check(p.prefill(cuda_lib), True, chunked=dtype == "bf16")


def test_step_is_the_same_alone_and_in_a_batch(cuda_lib):
    """A sequence's bits do not depend on what else is in the call (while the grid picks the same slices)."""
    c = Case(200, 2, 4, 128, 128, "bf16", T=4, seed=2)
    d = c.step(cuda_lib, True)
    half = Case(200, 2, 4, 128, 128, "bf16", T=4, seed=2, pad_seqs=range(0, 200, 2))
    e = half.step(cuda_lib, True)
    assert torch.equal(d["out"][1::2], e["out"][1::2])
    sl = c.slot[1::2].long()
    assert torch.equal(d["state"][sl.cuda()], e["state"][sl.cuda()])


@pytest.mark.parametrize("kind", ["step", "prefill"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_of_zero(cuda_lib, kind, dtype):
    """log_decay = -inf drops the state; a run of them, and the type's lowest value, do the same."""
    counts = [1, 5, 40, 200]
    c = Case(4, 1, 2, 64, 64, dtype, counts=counts, seed=9) if kind == "prefill" else Case(4, 1, 2, 64, 64, dtype, T=9, seed=9)
    g = c.tok["g"]
    if kind == "prefill":
        g[0], g[3, 0], g[10:14], g[60:200:17, 1], g[230] = -INF, -INF, -INF, -INF, torch.finfo(torch.float32).min
        c.check(c.prefill(cuda_lib), True, chunked=dtype == "bf16")
    else:
        g[0, 0], g[1, 8], g[2, 2:6, 1], g[3, 4] = -INF, -INF, -INF, torch.finfo(torch.float32).min
        c.check(c.step(cuda_lib, True), True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), INF, -INF])
def test_nonfinite_drafts_that_are_not_accepted_stay_out(cuda_lib, dtype, bad):
    """Rejected drafts, rows of padded sequences and rows past a packed sequence do not reach the state."""
    c = Case(4, 1, 2, 64, 64, dtype, counts=[3, 2, 4, 1], seed=4, pad_seqs=(2,)).add_prev(T=6, accept=[2, 0, 6, 5])
    for t in "kv":
        c.prev[t][0, 2:] = bad
        c.prev[t][1] = bad
        c.prev[t][3, 5:] = bad
        c.prev[t][2] = bad
    c.prev["g"][0, 2:], c.prev["g"][1] = bad, bad
    for t in "qkv":
        c.tok[t][c.cu[2]:c.cu[3]] = bad
    c.check(c.step(cuda_lib, False), False)


@pytest.mark.parametrize("kind", ["step", "prefill"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_nonfinite_tokens_do_not_reach_earlier_ones(cuda_lib, kind, dtype, where, bad):
    """A non-finite q, k or v at token t leaves every output before t as it is."""
    T, t = (300, 201) if kind == "prefill" else (8, 5)
    c = Case(1, 1, 2, 64, 64, dtype, counts=[T], seed=6)
    clean = Case(1, 1, 2, 64, 64, dtype, counts=[T], seed=6)
    c.tok[where][t, 0, 3] = bad
    run = (lambda x: x.prefill(cuda_lib)) if kind == "prefill" else (lambda x: x.step(cuda_lib, True))
    d, e = run(c), run(clean)
    assert torch.isfinite(d["out"][:t]).all()
    out, lim, _, _ = clean.expect(True, kind == "prefill" and dtype == "bf16")
    assert_within(d["out"][:t], out[:t], lim[:t], "out before the bad token")
    if where == "q":  # a bad query spoils its own output alone
        assert torch.equal(d["out"][t + 1:], e["out"][t + 1:])
        assert torch.equal(d["state"], e["state"])
    else:
        assert not torch.isfinite(d["out"][t]).all()


def test_initial_state_that_is_not_used_is_not_read(cuda_lib):
    c = Case(2, 1, 2, 64, 64, "bf16", T=2, seed=8, no_init=(0, 1))
    d = c.device()
    d["state"][c.slot.long().cuda()] = float("nan")
    c.check(c.step(cuda_lib, True, d), True)
    p = Case(2, 1, 2, 64, 64, "bf16", counts=[0, 140], seed=8, no_init=(0, 1))
    d = p.device()
    d["state"][p.slot.long().cuda()] = float("nan")
    p.check(p.prefill(cuda_lib, d), True, chunked=True)


def test_step_reports_bad_sequences_and_leaves_them(cuda_lib):
    c = Case(6, 1, 2, 64, 64, "bf16", counts=[2, 2, 2, 2, 2, 2], seed=1).add_prev(T=4, accept=[1, 5, -1, 2, 4, 0])
    d = c.device()
    d["slot"][3] = c.state.shape[0]
    d["cu"] = i32([0, 2, 4, 6, 8, 13, 12]).cuda()  # the last two spans: too long, reversed
    keep = {n: d[n].clone() for n in ("out", "state")}
    c.step(cuda_lib, True, d)
    assert d["err"].tolist() == [0, 4, 4, 1, 16, 16]
    out, lim, state, slim = c.expect(True, skip_seqs=(1, 2, 3, 4, 5))
    assert_within(d["out"], out, lim, "out")
    assert_within(d["state"], state, slim, "state")
    assert torch.equal(d["out"][2:], keep["out"][2:])


def test_step_on_another_stream(cuda_lib):
    c = Case(64, 2, 4, 128, 128, "bf16", T=4, seed=12).add_prev(T=4)
    d = c.device()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    c.step(cuda_lib, True, d, stream=st)
    c.check(d, True)


# ------------------------------------------------------------------------------------------- prompts


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,nq,nh,dk,dv", [
    ([1], 1, 1, 128, 128), ([127, 128, 129], 1, 2, 128, 128), ([0, 64, 1, 300], 2, 4, 128, 64), ([257, 5], 1, 3, 64, 128),
    ([65, 33, 2], 2, 2, 64, 64), ([200], 1, 2, 80, 56), ([130, 7], 1, 1, 16, 24), ([90], 1, 2, 12, 10),
    ([140, 20], 1, 1, 256, 200), ([1] * 40, 1, 2, 128, 128), ([515], 2, 2, 128, 96), ([33], 16, 48, 128, 128)])
def test_prefill_shapes(cuda_lib, counts, nq, nh, dk, dv, dtype):
    n = len(counts)
    c = Case(n, nq, nh, dk, dv, dtype, counts=counts, gain=nh % 2 == 0, skip=n % 2 == 1, seed=sum(counts),
             no_init=range(0, n, 2), decay=0.1)
    c.check(c.prefill(cuda_lib), True, chunked=dtype == "bf16")


@pytest.mark.parametrize("counts,nq,nh", [([3000], 1, 1), ([1, 2100, 900], 1, 2), ([2049], 2, 2)])
def test_prefill_long_prompts_split_over_their_length(cuda_lib, counts, nq, nh):
    """Few heads and long prompts: the length is split among blocks and joined; slow decays make every
    part matter to the ones after it."""
    c = Case(len(counts), nq, nh, 64, 64, "bf16", counts=counts, gain=True, seed=7, decay=0.002)
    c.check(c.prefill(cuda_lib), True, chunked=True)


@pytest.mark.parametrize("dtype,counts,nq,nh,dk,dv", [
    ("f32", [900], 1, 1, 64, 64), ("f32", [1, 333, 600, 0], 1, 2, 128, 32), ("f32", [97, 98], 2, 2, 20, 128),
    ("f32", [2000], 1, 3, 128, 128), ("bf16", [500, 77], 1, 1, 128, 136)])
def test_prefill_recurrent_prompts_split_over_their_length(cuda_lib, dtype, counts, nq, nh, dk, dv):
    """Prompts the chunked kernel does not take, cut into pieces; slow decays make every piece matter."""
    c = Case(len(counts), nq, nh, dk, dv, dtype, counts=counts, gain=True, seed=17, decay=0.003, no_init=(len(counts) - 1,))
    c.check(c.prefill(cuda_lib), True)


def test_prefill_own_workspace(cuda_lib):
    """A caller's workspace of the reported size will do, a smaller one is refused before anything is launched."""
    c = Case(1, 1, 2, 64, 64, "f32", counts=[700], seed=18)
    d = c.device()
    need = cuda_lib.linattn_workspace(d["q"], d["k"], d["v"], d["g"], d["state"], d["out"], d["cu"], max_seqlen=700)
    assert need > 0
    with pytest.raises(cuda_lib.CvError) as e:
        c.prefill(cuda_lib, d, workspace=torch.empty(need - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -13 and bool((d["out"] == SENT).all())
    c.check(c.prefill(cuda_lib, d, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")), True)


def test_prefill_padded_and_bad_spans(cuda_lib):
    c = Case(5, 1, 2, 64, 64, "bf16", counts=[40, 150, 30, 200, 10], seed=3, pad_seqs=(1,))
    d = c.device()
    d["cu"] = i32([0, 40, 190, 220, 420, 430]).cuda()
    d["slot"][4] = c.state.shape[0] + 5
    c.prefill(cuda_lib, d, max_seqlen=199)
    c.check(d, True, chunked=True, err=[0, 0, 0, 16, 1], skip_seqs=(3, 4))


def test_prefill_equals_its_parts(cuda_lib):
    """A prompt in two calls, the second from the first one's state, equals the prompt in one (fp32: the
    recurrent order is the same; bf16 within the bounds)."""
    c = Case(1, 2, 4, 64, 64, "bf16", counts=[230], gain=True, seed=5)
    d = c.device()
    for lo, hi in ((0, 131), (131, 230)):
        cuda_lib.linattn_prefill(d["q"][lo:hi], d["k"][lo:hi], d["v"][lo:hi], d["g"][lo:hi], d["state"], d["out"][lo:hi],
                                 i32([0, hi - lo]).cuda(), max_seqlen=hi - lo, gain=d["b"][lo:hi], scale=c.scale,
                                 cache_idx=d["slot"], err=d["err"])
    torch.cuda.synchronize()
    c.check(d, True, chunked=True)


@pytest.mark.parametrize("counts,nq,nh,dk,dv", [
    ([700, 129, 1500], 1, 4, 128, 128),
    ([(37 * i * i) % 2900 + 1 for i in range(30)], 2, 6, 64, 128),  # several units a block, of very different lengths
    ([(53 * i * i) % 1700 for i in range(12)], 4, 24, 128, 64)])
def test_prefill_repeats_bit_for_bit(cuda_lib, counts, nq, nh, dk, dv):
    """The roles of the chunked kernel hand work on through barriers alone: a missed one shows as a difference."""
    c = Case(len(counts), nq, nh, dk, dv, "bf16", counts=counts, seed=21, gain=True)
    first = c.prefill(cuda_lib)
    assert first["err"].tolist() == [0] * len(counts)
    for _ in range(6):
        d = c.prefill(cuda_lib)
        assert torch.equal(d["out"], first["out"]) and torch.equal(d["state"], first["state"])


@pytest.mark.parametrize("dtype,counts,nq,nh,dk,dv", [
    ("bf16", [3000, 2670, 2171, 118, 1907, 1020, 2658, 212], 4, 8, 64, 64),  # more pieces than SMs
    ("bf16", [0, 2300, 130, 0, 700], 1, 3, 128, 128),
    ("f32", [428, 1257, 0, 115], 8, 24, 128, 128),
    ("f32", [91, 148, 18, 284, 226, 93, 63, 49, 0, 252, 158, 126], 1, 4, 128, 88)])
def test_prefill_cut_ragged_prompts(cuda_lib, dtype, counts, nq, nh, dk, dv):
    """Pieces of one prompt run in any order: the first reads the state that the last one writes."""
    c = Case(len(counts), nq, nh, dk, dv, dtype, counts=counts, seed=23, gain=True)
    first = c.prefill(cuda_lib)
    assert first["err"].tolist() == [0] * len(counts)
    c.check(first, True, chunked=dtype == "bf16")
    for _ in range(8):
        d = c.prefill(cuda_lib)
        assert torch.equal(d["out"], first["out"]) and torch.equal(d["state"], first["state"])


def test_prefill_on_another_stream(cuda_lib):
    c = Case(2, 1, 2, 128, 128, "bf16", counts=[900, 333], seed=22)
    d = c.device()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    c.prefill(cuda_lib, d, stream=st)
    c.check(d, True, chunked=True)


def test_step_decays_multiply_exactly_once(cuda_lib):
    """Closed form: k = v = e_1, q = e_1, constant decay a: out_t = sum_{u<=t} a^(t-u)."""
    T, a = 6, 0.5
    q = torch.zeros(1, T, 1, 8, device="cuda")
    q[..., 0] = 1
    out, state = torch.zeros(1, T, 1, 8, device="cuda"), torch.zeros(1, 1, 8, 8, device="cuda")
    g = torch.full((1, T, 1), math.log(a), device="cuda")
    cuda_lib.linattn_step(q, q, q, g, state, out, scale=1.0, update_state=True)
    want = torch.tensor([sum(a ** (t - u) for u in range(t + 1)) for t in range(T)])
    assert torch.allclose(out[0, :, 0, 0].cpu(), want, rtol=1e-6, atol=0)
    assert torch.allclose(state[0, 0, 0, 0].cpu(), want[-1], rtol=1e-6, atol=0)
    assert float(out[..., 1:].abs().max()) == 0 and float(state.flatten()[1:].abs().max()) == 0
