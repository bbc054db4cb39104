"""Attention of drafted tokens over a paged cache, against the softmax in 64 bits.  Every place of the cache that a call has no
business with holds NaN, and so do the page table's entries past those in use (as numbers of no page)."""
from __future__ import annotations

import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(lens, counts, T, n_kv, G, d, page, dtype, tree=False, ragged=False, seed=0, pad=(), slack=2, head_major=False):
    """Inputs on the CPU: sequences with lens cached tokens and counts drafts."""
    g = torch.Generator().manual_seed(seed)
    n, H = len(lens), n_kv * G
    need = [-(-(L + c) // page) for L, c in zip(lens, counts)]
    rows = n + 1
    slots = torch.randperm(rows, generator=g)[:n].int()
    for s in pad:
        slots[s] = -1
    n_pages = sum(need) + slack
    order = torch.randperm(n_pages, generator=g).int()
    table = torch.full((rows, max(max(need), 1) + 1), 10 ** 9, dtype=torch.int32)
    shape = (n_pages, n_kv, page, d) if head_major else (n_pages, page, n_kv, d)
    k, v = torch.full(shape, float("nan"), dtype=dtype), torch.full(shape, float("nan"), dtype=dtype)
    if head_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    at = 0
    for s in range(n):
        if slots[s] < 0:
            continue
        table[slots[s], :need[s]] = order[at:at + need[s]]
        at += need[s]
        for x in range(lens[s] + counts[s]):
            pg = int(table[slots[s], x // page])
            k[pg, x % page] = torch.randn(n_kv, d, generator=g).to(dtype)
            v[pg, x % page] = torch.randn(n_kv, d, generator=g).to(dtype)
    parents = []
    for c in counts:
        parents.append([-1 if t == 0 else int(torch.randint(-1 if tree == "forest" else 0, t, (1,), generator=g)) for t in range(c)]
                       if tree else ref.chain(c))
    lead = (sum(counts),) if ragged else (n, T)
    # q and out as slices of wider rows
    q = torch.randn(*lead, H + 1, d + 8, generator=g).to(dtype)[..., :H, :d]
    cu = torch.tensor([0] + list(counts)).cumsum(0).int() if ragged else None
    parent = None
    if tree:
        flat = [p for seq in parents for p in seq]
        parent = torch.tensor(flat, dtype=torch.int32).view(lead)
    return dict(q=q, k=k, v=v, table=table, slots=slots, lens=lens, counts=counts, T=T, cu=cu, parent=parent, parents=parents)


def on_gpu(t):
    if t is None:
        return None
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda") if t.numel() else t.cuda()
    out.copy_(t)
    return out


def call(cv, x, scale=None, **kw):
    """Runs the call; out starts at 7 everywhere."""
    cache = cv.PagedCache(on_gpu(x["k"]), on_gpu(x["v"]), x["table"].cuda())
    q = on_gpu(x["q"])
    out = torch.full((*q.shape[:-1], q.shape[-1] + 8), 7.0, dtype=q.dtype, device="cuda")[..., :q.shape[-1]]
    err = torch.full((len(x["lens"]),), -7, dtype=torch.int32, device="cuda")
    cv.tree_attention(q, out, cache, torch.tensor(x["lens"], dtype=torch.int32).cuda(), parent=on_gpu(x["parent"]),
                      cu_draft=on_gpu(x["cu"]), T=x["T"], cache_idx=x["slots"].cuda(), err=err, scale=scale, **kw)
    torch.cuda.synchronize()
    return out.cpu(), err.cpu().tolist()


def rows_of(x, out, s):
    """Sequence s's rows of a packed or batched tensor."""
    if x["cu"] is not None:
        return out[int(x["cu"][s]):int(x["cu"][s + 1])]
    return out[s, :x["counts"][s]]


def check(x, out, err, scale=None, flagged=()):
    d = x["q"].shape[-1]
    for s, L in enumerate(x["lens"]):
        got = rows_of(x, out, s).double()
        if x["slots"][s] < 0 or s in flagged:
            assert bool((got == 7).all()), f"sequence {s} was written"
            continue
        assert err[s] == 0
        c = x["counts"][s]
        if c == 0:
            continue
        row = x["table"][int(x["slots"][s])]
        K, V = ref.gather(x["k"], row, L + c), ref.gather(x["v"], row, L + c)
        want, size, top = ref.attention(rows_of(x, x["q"], s).double(), K, V, L, x["parents"][s], scale or d ** -0.5)
        bound = ref.attention_bound(x["q"].dtype, want, size, top, L + c, d)
        off = (got - want).abs()
        assert bool((off <= bound).all()), f"sequence {s}: {float((off / bound).max()):.2f} times the bound"


SHAPES = [  # n_kv, G, d, page
    (2, 4, 128, 16), (1, 1, 64, 16), (4, 8, 64, 32), (2, 6, 256, 16), (1, 16, 128, 64), (3, 3, 96, 128), (1, 5, 192, 8),
    (2, 2, 40, 256), (1, 4, 17, 16), (2, 1, 128, 5), (1, 2, 1, 1), (1, 40, 64, 16), (1, 130, 16, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_kv,G,d,page", SHAPES)
def test_shapes(cuda_lib, n_kv, G, d, page, dtype):
    x = make([0, 1, 37, 300], [3] * 4, 3, n_kv, G, d, page, dtype, tree=True, pad=(1,))
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 7, 16, 33, 128])
@pytest.mark.parametrize("tree", [False, True, "forest"])
def test_draft_counts(cuda_lib, T, tree, dtype):
    x = make([0, 65, 127, 128, 500], [T] * 5, T, 2, 2, 64, 16, dtype, tree=tree, seed=T)
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tree", [False, True])
def test_ragged(cuda_lib, tree, dtype):
    counts = [1, 17, 0, 5, 128, 2, 0, 9]
    x = make([700, 3, 50, 0, 129, 1030, 0, 64], counts, 128, 2, 4, 128, 16, dtype, tree=tree, ragged=True, pad=(3,))
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [1, 63, 64, 126, 127, 128, 129, 255, 5000, 20001])
def test_one_sequence_cut_over_all_blocks(cuda_lib, L, dtype):
    x = make([L], [2], 2, 1, 4, 128, 16, dtype)
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences(cuda_lib, dtype):
    """More sequences than a block has threads; empty and padded ones in long runs."""
    n = 700
    lens = [(i * 37) % 50 for i in range(n)]
    counts = [0 if i % 5 == 0 or 200 < i < 450 else 1 + i % 2 for i in range(n)]
    x = make(lens, counts, 2, 1, 2, 64, 16, dtype, ragged=True, pad=tuple(range(460, 520)))
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_heads_before_rows_in_a_page_and_a_scale(cuda_lib, dtype):
    x = make([90, 200], [4, 4], 4, 3, 2, 128, 32, dtype, head_major=True)
    check(x, *call(cuda_lib, x, scale=0.5), scale=0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_scores(cuda_lib, dtype):
    """Scores of hundreds that rise along the cache: every tile moves the maximum."""
    x = make([1000], [3], 3, 1, 4, 64, 16, dtype)
    page = x["k"].shape[1]
    row = x["table"][int(x["slots"][0])]
    for j in range(1003):
        x["k"][int(row[j // page]), j % page] *= 0.02 * j
    check(x, *call(cuda_lib, x))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("L", [5, 100, 126])
def test_values_that_are_not_finite_stay_where_they_are_seen(cuda_lib, bad, L, dtype):
    """A draft's v (or k) that is not finite reaches its descendants and nobody else."""
    for which in "kv":
        x = make([L], [9], 9, 1, 3, 64, 16, dtype, tree=True, seed=3)
        page = x["k"].shape[1]
        row = x["table"][int(x["slots"][0])]
        at = (int(row[(L + 4) // page]), (L + 4) % page)
        x[which][at[0], at[1], 0, 7] = bad
        out, err = call(cuda_lib, x)
        assert err == [0]
        seen = ref.ancestors(x["parents"][0])
        K, V = ref.gather(x["k"], row, L + 9), ref.gather(x["v"], row, L + 9)
        K, V = K.nan_to_num(0, 0, 0), V.nan_to_num(0, 0, 0)
        want, size, top = ref.attention(x["q"][0].double(), K, V, L, x["parents"][0], 64 ** -0.5)
        bound = ref.attention_bound(dtype, want, size, top, L + 9, 64)
        for t in range(9):
            got = out[0, t].double()
            if 4 not in seen[t]:
                assert bool(((got - want[t]).abs() <= bound[t]).all())
            elif which == "v":
                assert bool((~torch.isfinite(got[:, 7])).all())
                if bad == bad:
                    assert bool((got[:, 7] == bad).all())
                keep = torch.arange(64) != 7
                assert bool(((got - want[t]).abs() <= bound[t])[:, keep].all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_of_minus_infinity(cuda_lib, dtype):
    """A cached key far below the others' scores has no weight; where every seen score is minus infinity the result is NaN."""
    x = make([300], [2], 2, 1, 1, 64, 16, dtype)
    x["q"][...] = 1.0
    page = x["k"].shape[1]
    row = x["table"][int(x["slots"][0])]
    for j in range(200):
        x["k"][int(row[j // page]), j % page, 0, 0] = -float("inf")
    out, err = call(cuda_lib, x)
    K, V = ref.gather(x["k"], row, 302), ref.gather(x["v"], row, 302)
    want, size, _ = ref.attention(x["q"][0].double(), K, V, 300, x["parents"][0], 0.125)
    _, _, top = ref.attention(x["q"][0].double(), K[200:], V[200:], 100, x["parents"][0], 0.125)
    assert bool(((out[0].double() - want).abs() <= ref.attention_bound(dtype, want, size, top, 302, 64)).all())
    for j in range(302):
        x["k"][int(row[j // page]), j % page, 0, 0] = -float("inf")
    out, err = call(cuda_lib, x)
    assert err == [0] and bool(torch.isnan(out).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_flags(cuda_lib, dtype):
    """A slot, a length, a page or a parent that is not there flags its sequence and leaves its rows alone."""
    x = make([40, 50, 60, 70, 900, 30], [4] * 6, 4, 2, 2, 64, 16, dtype, tree=True)
    row = int(x["slots"][3])
    x["slots"][0] = x["table"].shape[0]
    x["lens"][1] = -1
    x["table"][row, 4] = x["k"].shape[0]
    x["table"][int(x["slots"][4]), 20] = -1
    x["parent"][5, 2] = 2
    out, err = call(cuda_lib, x)
    assert err == [1, 64, 0, 128, 128, 32]
    lens = list(x["lens"])
    for s in (0, 1, 3, 4, 5):
        assert bool((out[s] == 7).all())
    x["lens"] = lens
    check(x, out, err, flagged=(0, 1, 3, 4, 5))
    x["lens"][2] = x["table"].shape[1] * 16 - 3
    assert call(cuda_lib, x)[1][2] == 64


def test_bad_spans(cuda_lib):
    x = make([40, 50, 60], [4, 4, 4], 4, 1, 2, 64, 16, BF, ragged=True)
    x["cu"] = torch.tensor([0, 4, 3, 12], dtype=torch.int32)
    out, err = call(cuda_lib, x)
    assert err == [0, 16, 16]
    assert bool((out[4:] == 7).all())


def test_the_same_bits_every_time_and_in_a_graph(cuda_lib):
    cv = cuda_lib
    x = make([3000, 10, 777], [5, 5, 5], 5, 2, 4, 128, 16, BF, tree=True)
    cache = cv.PagedCache(on_gpu(x["k"]), on_gpu(x["v"]), x["table"].cuda())
    q, lens, par = on_gpu(x["q"]), torch.tensor(x["lens"], dtype=torch.int32).cuda(), on_gpu(x["parent"])
    slots = x["slots"].cuda()
    outs = []
    for _ in range(3):
        out = torch.zeros(q.shape, dtype=BF, device="cuda")
        cv.tree_attention(q, out, cache, lens, parent=par, cache_idx=slots)
        outs.append(out)
    graph, out = torch.cuda.CUDAGraph(), torch.zeros(q.shape, dtype=BF, device="cuda")
    with torch.cuda.graph(graph):
        cv.tree_attention(q, out, cache, lens, parent=par, cache_idx=slots)
    # a replay reads the lengths of its time
    graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, out)
    lens.sub_(1)
    graph.replay()
    eager = torch.zeros_like(out)
    cv.tree_attention(q, eager, cache, lens, parent=par, cache_idx=slots)
    torch.cuda.synchronize()
    assert torch.equal(out, eager) and not torch.equal(out, outs[0])


def test_streams_and_a_workspace_of_ones_own(cuda_lib):
    cv = cuda_lib
    x = make([2000, 400], [3, 3], 3, 2, 4, 128, 16, BF)
    cache = cv.PagedCache(on_gpu(x["k"]), on_gpu(x["v"]), x["table"].cuda())
    q, lens, slots = on_gpu(x["q"]), torch.tensor(x["lens"], dtype=torch.int32).cuda(), x["slots"].cuda()
    outs = [torch.zeros(q.shape, dtype=BF, device="cuda") for _ in range(4)]
    need = cv.tree_attention_workspace(q, outs[0], cache, lens, cache_idx=slots)
    assert need > 0
    torch.cuda.synchronize()
    cv.tree_attention(q, outs[0], cache, lens, cache_idx=slots)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, out in zip(streams, outs[1:]):
        cv.tree_attention(q, out, cache, lens, cache_idx=slots, stream=st)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    cv.tree_attention(q, outs[3], cache, lens, cache_idx=slots, workspace=ws)
    torch.cuda.synchronize()
    for out in outs[1:]:
        assert torch.equal(out, outs[0])
    with pytest.raises(cv.CvError):
        cv.tree_attention(q, outs[3], cache, lens, cache_idx=slots, workspace=ws[:need - 256])
