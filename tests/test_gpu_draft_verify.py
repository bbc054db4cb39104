"""Verification of drafted tokens, against the walk and the sums in 64 bits: whole numbers, equal."""
from __future__ import annotations

import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(counts, T, vocab, dtype, mode, ragged=False, seed=0, pad=()):
    g = torch.Generator().manual_seed(seed)
    n = len(counts)
    seqs = []
    for c in counts:
        p = ref.decaying(c, vocab, g).to(dtype)
        q = torch.softmax(p.float().clamp(min=1e-30).log() + 0.7 * torch.randn(c, vocab, generator=g), -1).to(dtype)
        parent = ref.chain(c) if mode != "tree" else [-1] + [int(torch.randint(max(0, t - 3), t, (1,), generator=g)) for t in range(1, c)]
        of = q if mode == "q" else p
        tok = [int(torch.randint(vocab, (1,), generator=g))]
        drawn = q.clone()
        for t in range(1, c):
            tok.append(int(torch.multinomial(of[parent[t]].float(), 1, generator=g)))
            drawn[t] = q[parent[t]]
        seqs.append(dict(p=p, q=drawn if mode == "q" else None, tok=tok, parent=parent, u=torch.rand(T + 1, generator=g)))
    slots = torch.arange(n, dtype=torch.int32)
    for s in pad:
        slots[s] = -1

    def put(name, like):
        if seqs[0][name] is None:
            return None
        rows = [torch.as_tensor(s[name]) for s in seqs]
        if ragged:
            return torch.cat(rows).to(like)
        return torch.stack(rows).to(like)

    return dict(seqs=seqs, counts=counts, T=T, p=put("p", dtype), q=put("q", dtype), tok=put("tok", torch.int32),
                parent=put("parent", torch.int32) if mode == "tree" else None, u=torch.stack([s["u"] for s in seqs]), slots=slots,
                cu=torch.tensor([0] + list(counts)).cumsum(0).int() if ragged else None)


def call(cv, x, p=None, q=None):
    n, T = len(x["counts"]), x["T"]
    dev = lambda t: t.cuda() if t is not None else None  # noqa: E731
    full = lambda *s: torch.full(s, -5, dtype=torch.int32, device="cuda")  # noqa: E731
    accept, node, out, path, err = full(n), full(n), full(n, T), full(n, T), full(n)
    cv.draft_verify(dev(x["p"]) if p is None else p, dev(x["tok"]), dev(x["u"]), accept, out,
                    draft_probs=dev(x["q"]) if q is None else q, parent=dev(x["parent"]), path=path, accept_node=node,
                    cu_draft=dev(x["cu"]), T=T, cache_idx=dev(x["slots"]), err=err)
    torch.cuda.synchronize()
    return tuple(t.cpu() for t in (accept, node, out, path, err))


def check(x, got, flagged=()):
    accept, node, out, path, err = got
    for s, seq in enumerate(x["seqs"]):
        if x["slots"][s] < 0 or s in flagged:
            assert accept[s] == node[s] == -5 and bool((out[s] == -5).all()) and bool((path[s] == -5).all())
            continue
        want, new = ref.verify(seq["p"], seq["tok"], seq["u"], seq["parent"], seq["q"])
        pad = [-1] * (x["T"] - len(want))
        assert err[s] == 0
        assert path[s].tolist() == want + pad
        assert accept[s] == len(want) and node[s] == want[-1] + 1
        assert out[s].tolist() == [seq["tok"][t] for t in want[1:]] + [new] + pad


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("mode", ["q", "plain", "tree"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 127, 1000, 4099, 50257])
def test_vocabularies(cuda_lib, vocab, mode, dtype):
    x = make([5] * 12, 5, vocab, dtype, mode, seed=vocab, pad=(3,))
    check(x, call(cuda_lib, x))


@pytest.mark.parametrize("mode", ["q", "plain", "tree"])
@pytest.mark.parametrize("T", [1, 2, 16, 128])
def test_draft_counts(cuda_lib, T, mode):
    x = make([T] * 6, T, 300, F32, mode, seed=T)
    check(x, call(cuda_lib, x))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("mode", ["q", "plain", "tree"])
def test_ragged(cuda_lib, mode, dtype):
    x = make([1, 9, 4, 17, 2, 6], 17, 1111, dtype, mode, ragged=True, pad=(2,))
    check(x, call(cuda_lib, x))


def test_no_drafts_at_all_is_a_span_that_is_flagged(cuda_lib):
    x = make([3, 4], 4, 50, F32, "plain", ragged=True)
    x["cu"] = torch.tensor([0, 3, 3], dtype=torch.int32)
    got = call(cuda_lib, x)
    assert got[4].tolist() == [0, 16] and got[0][1] == -5


def test_ends_of_the_uniforms(cuda_lib):
    """0 takes the first token with any weight, the largest below 1 the last; numbers outside count as the ends."""
    V = 1000
    p = torch.zeros(6, 1, V)
    p[:, 0, 17], p[:, 0, 500], p[:, 0, 901] = 0.25, 0.5, 0.25
    x = dict(counts=[1] * 6, T=1, p=p, q=None, tok=torch.zeros(6, 1, dtype=torch.int32), parent=None, cu=None,
             u=torch.tensor([[0, 0.0], [0, 0.25], [0, 0.75], [0, 1.0], [0, -3.0], [0, float("nan")]]), slots=torch.arange(6).int())
    assert call(cuda_lib, x)[2].flatten().tolist() == [17, 500, 901, 901, 17, 17]


def test_ties_twins_and_nothing_left(cuda_lib):
    V = 64
    p = torch.zeros(5, 4, V)
    p[..., 3] = 0.5
    p[..., 9] = 0.5
    tok = torch.tensor([[1, 3, 3, 9]] * 5, dtype=torch.int32)
    parent = torch.tensor([[-1, 0, 0, 0]] * 4 + [[-1, 0, 0, -1]], dtype=torch.int32)
    u = torch.full((5, 5), 0.6)
    u[0, 0] = 0.5          # not below 0.5: the first child falls, its twin is passed over, the third stands
    u[1, 0] = 0.4999
    u[2, 0] = 0.9999
    u[3, 0] = 0.99999994
    p[3, 0, 9] = 0.4999    # the children's masses end below the draw: nothing is left but the row itself
    u[4, 0] = 0.7          # token 3 is nobody's child: the rest of the row is sampled
    x = dict(counts=[4] * 5, T=4, p=p, q=None, tok=tok, parent=parent, cu=None, u=u, slots=torch.arange(5).int())
    accept, node, out, path, err = call(cuda_lib, x)
    assert err.tolist() == [0] * 5
    assert path[:, 1].tolist() == [3, 1, 3, -1, -1]
    assert node.tolist() == [4, 2, 4, 1, 1]
    assert out[3, 0] == 9 and out[4, 0] == 9


def test_equal_distributions_accept_and_fall_back_to_the_target(cuda_lib):
    """p = q: every draft below its probability stands; where q is above p everywhere it can be, the row itself is sampled."""
    V = 500
    g = torch.Generator().manual_seed(0)
    p = ref.decaying(3, V, g).view(1, 3, V)
    q = torch.cat([p[:, :1], p[:, :1], p[:, 1:2]], 1)
    tok = torch.tensor([[0, int(p[0, 0].argmax()), int(p[0, 1].argmax())]], dtype=torch.int32)
    x = dict(counts=[3], T=3, p=p, q=q, tok=tok, parent=None, cu=None, u=torch.full((1, 4), 0.999), slots=torch.zeros(1).int(),
             seqs=[dict(p=p[0], q=q[0], tok=tok[0].tolist(), parent=[-1, 0, 1], u=torch.full((4,), 0.999))])
    check(x, call(cuda_lib, x))
    q2 = (q * 1.5).contiguous()
    x["q"], x["seqs"][0]["q"] = q2, q2[0]
    check(x, call(cuda_lib, x))
    assert call(cuda_lib, x)[0][0] == 1


def test_values_that_are_no_probabilities(cuda_lib):
    """NaN, negative numbers and zero count as zero; an all-zero row and rows that add up to 4 and more are flagged."""
    V = 300
    p = torch.full((4, 1, V), 1.0 / V)
    p[0, 0, :150] = float("nan")
    p[0, 0, 150:200] = -1.0
    p[1] = 0
    p[2] = 0.5
    p[3, 0, 5] = float("inf")
    p[3, 0, 6] = float("inf")
    x = dict(counts=[1] * 4, T=1, p=p, q=None, tok=torch.zeros(4, 1, dtype=torch.int32), parent=None, cu=None, u=torch.zeros(4, 2),
             slots=torch.arange(4).int())
    accept, _, out, _, err = call(cuda_lib, x)
    assert err.tolist() == [0, 512, 512, 512] and out[0, 0] == 200 and accept.tolist() == [1, -5, -5, -5]


def test_flags(cuda_lib):
    x = make([5] * 4, 5, 100, F32, "tree", seed=1)
    x["tok"][0, 3] = 100
    x["tok"][1, 0] = -4  # token 0 is not looked up
    x["parent"][2, 0] = 0
    x["parent"][3, 4] = 4
    for s in range(4):
        x["seqs"][s]["tok"] = x["tok"][s].tolist()
    got = call(cuda_lib, x)
    assert got[4].tolist() == [256, 0, 32, 32]
    check(x, got, flagged=(0, 2, 3))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("mode", ["q", "plain"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rows_at_any_address(cuda_lib, shift, mode, dtype):
    """Rows of odd strides, each at another offset from a 16-byte boundary."""
    x = make([4] * 8, 4, 777, dtype, mode, seed=9)

    def strided(t, more):
        if t is None:
            return None
        flat = torch.full((8 * 4 * (777 + more) + 16,), 9.0, dtype=dtype, device="cuda")
        view = flat[shift:].as_strided(t.shape, (4 * (777 + more), 777 + more, 1), flat.storage_offset() + shift)
        view.copy_(t)
        return view

    check(x, call(cuda_lib, x, p=strided(x["p"], 3), q=strided(x["q"], 5)))


def test_sampling_follows_the_target(cuda_lib):
    """Drafts from another distribution leave the target's: of 20,000 first tokens each value's share is its probability within
    6 standard deviations (8 values: a chance of 1e-8)."""
    n, V = 20000, 8
    g = torch.Generator().manual_seed(0)
    p = torch.tensor([0.30, 0.20, 0.15, 0.12, 0.10, 0.08, 0.04, 0.01]).expand(n, 2, V).contiguous()
    q = torch.tensor([0.05, 0.40, 0.05, 0.10, 0.10, 0.20, 0.05, 0.05]).expand(n, 2, V).contiguous()
    tok = torch.zeros(n, 2, dtype=torch.int32)
    tok[:, 1] = torch.multinomial(q[:, 0], 1, generator=g)[:, 0].int()
    x = dict(counts=[2] * n, T=2, p=p, q=q, tok=tok, parent=None, cu=None, u=torch.rand(n, 3, generator=g), slots=torch.arange(n).int())
    for with_q in (True, False):
        if not with_q:
            x["q"] = None
        first = call(cuda_lib, x)[2][:, 0]
        share = torch.bincount(first.long(), minlength=V).double() / n
        want = p[0, 0].double()
        assert bool(((share - want).abs() <= 6 * torch.sqrt(want * (1 - want) / n)).all())
