"""A run of the attention layers' operators as a serving program makes it: prompts, then steps of drafted trees with pages reserved,
attention, verification, and the accepted path compacted, against one long causal attention over the accepted tokens."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import attn_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [0, 1])
def test_attention_layer(cuda_lib, seed):
    """Steps of trees against one prompt of the accepted tokens.  Keys and values are the same bits, so only the order of sums and the
    rounding of the weights and outputs to bf16 differ: each side is off by at most 2^-8 of an output and 2^-8 of the mean size of the
    values that it is made of (the sums themselves by 1 % of that), neither above the largest value."""
    import attention_layer
    d_out, top, d_cache = attention_layer.main(seed=seed)
    assert d_cache == 0
    assert d_out <= 2 * (2.0 ** -8 + 2.0 ** -8) * top * 1.01


def layer(cv, n, T, H, n_kv, d, page, vocab, seed):
    """Buffers of one step of n sequences of T drafts."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    table = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
    held, refs = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n * 8 + 3, dtype=torch.int32, device="cuda")
    k = torch.zeros(n * 8 + 3, page, n_kv, d, dtype=torch.bfloat16, device="cuda")
    half = torch.arange(8 * page, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    parent = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 5][:T]] * n, dtype=torch.int32, device="cuda")
    return dict(cache=cv.PagedCache(k, torch.zeros_like(k), table, held=held, refs=refs), x=rnd(n, T, (H + 2 * n_kv) * d),
                cs=torch.cat([half.cos(), half.sin()], 1).float(), len=ints(n), want=ints(n), q=rnd(n, T, H, d), out=rnd(n, T, H, d),
                probs=torch.softmax(3 * torch.randn(n, T, vocab, generator=g, device="cuda"), -1), parent=parent,
                tok=torch.randint(vocab, (n, T), generator=g, device="cuda").int(), u=torch.rand(n, T + 1, generator=g, device="cuda"),
                accept=ints(n), node=ints(n), new=ints(n, T), path=ints(n, T), new_len=ints(n))


def step(cv, b, T, H, n_kv, d, stream=None):
    """reserve, norms and rotation, attention, verification, compaction, and the tail's pages back; no host read between."""
    torch.add(b["len"], T, out=b["want"])
    cv.cache_reserve(b["cache"], b["want"], stream=stream)
    x = b["x"]
    q = x[..., :H * d].unflatten(-1, (H, d))
    k, v = (x[..., (H + i * n_kv) * d:(H + (i + 1) * n_kv) * d].unflatten(-1, (n_kv, d)) for i in range(2))
    cv.qk_norm_rope(q, k, b["q"], v=v, cos_sin=b["cs"], cache=b["cache"], cache_len=b["len"], stream=stream)
    cv.tree_attention(b["q"], b["out"], b["cache"], b["len"], parent=b["parent"], stream=stream)
    cv.draft_verify(b["probs"], b["tok"], b["u"], b["accept"], b["new"], parent=b["parent"], path=b["path"], accept_node=b["node"],
                    stream=stream)
    cv.cache_compact(b["cache"], b["len"], b["path"], b["accept"], new_len=b["new_len"], stream=stream)
    b["len"].copy_(b["new_len"])
    cv.cache_free(b["cache"], b["len"], stream=stream)


def test_a_captured_step_replays_what_eager_steps_do(cuda_lib):
    """Three eager steps against three replays of a captured one: equal caches, tables, lengths and tokens."""
    cv, shape = cuda_lib, (8, 8, 2, 64)
    a, b = (layer(cv, 3, shape[0], shape[1], shape[2], shape[3], 16, 100, 5) for _ in range(2))
    for _ in range(3):
        step(cv, a, *shape)
    graph = torch.cuda.CUDAGraph()
    step(cv, layer(cv, 3, shape[0], shape[1], shape[2], shape[3], 16, 100, 6), *shape)  # (kernels loaded before the capture)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(cv, b, *shape)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name in ("len", "accept", "node", "new", "path", "out"):
        assert torch.equal(a[name], b[name]), name
    for x, y in zip(a["cache"]._tensors(), b["cache"]._tensors()):
        assert torch.equal(x, y)
    assert bool((a["len"] >= 3).all()) and int(a["cache"].refs.sum()) == int(a["cache"].held.sum())


def test_two_captured_graphs_run_at_once(cuda_lib):
    """Graphs captured one after the other on streams of their own have workspaces of their own."""
    cv, shape = cuda_lib, (8, 8, 2, 64)
    sets = [layer(cv, 40, shape[0], shape[1], shape[2], shape[3], 16, 100, s) for s in (7, 8)]
    want = [layer(cv, 40, shape[0], shape[1], shape[2], shape[3], 16, 100, s) for s in (7, 8)]
    for w in want:
        for _ in range(4):
            step(cv, w, *shape)
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in sets], []
    for s, b in zip(streams, sets):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            step(cv, b, *shape)
    for _ in range(4):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for w, b in zip(want, sets):
        for name in ("len", "accept", "new", "path", "out"):
            assert torch.equal(w[name], b[name]), name


def test_verify_hands_on_to_the_commits(cuda_lib):
    """accept_len and accept_node are what cv_conv_commit takes: the window after it is that of the last accepted token."""
    cv, n, T, dim, V = cuda_lib, 6, 5, 64, 50
    g = torch.Generator().manual_seed(3)
    parent = [-1, 0, 0, 1, 2]
    p = ref.decaying(n * T, V, g).view(n, T, V)
    tok = torch.stack([torch.multinomial(p[:, max(q, 0)], 1, generator=g)[:, 0] for q in parent], 1).int()
    x, state = torch.randn(n, T, dim, generator=g).cuda(), torch.randn(n, dim, 3, generator=g).cuda()
    before, w = state.clone(), torch.randn(dim, 4, generator=g).cuda()
    win, out = torch.zeros(n, T, dim, 3, device="cuda"), torch.zeros(n, T, dim, device="cuda")
    par = torch.tensor([parent] * n, dtype=torch.int32).cuda()
    cv.conv_verify(x, state, w, None, out, win, layout="dense", qk_channels=0, head_dim=8, parent=par)
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    accept, node, new, path = ints(n), ints(n), ints(n, T), ints(n, T)
    cv.draft_verify(p.cuda(), tok.cuda(), torch.rand(n, T + 1, generator=g).cuda(), accept, new, parent=par, path=path, accept_node=node)
    cv.conv_commit(state, win, node, layout="dense", T=T, width=4)
    torch.cuda.synchronize()
    for s in range(n):
        seen = [t for t in path[s].tolist() if t >= 0]
        assert len(seen) == accept[s] and seen == ref.ancestors(parent)[seen[-1]]
        want = torch.cat([before[s], x[s, seen].T], 1)[:, -3:]
        assert torch.equal(state[s], want)
