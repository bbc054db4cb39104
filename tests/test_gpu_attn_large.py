"""Caches and probabilities of more than 2^31 elements: the far end gives what the same rows give in small tensors."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def far(cuda_lib):
    """A cache of 2.3e9 elements whose last pages are used, a small one of the same rows, and their tables."""
    cv = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(0)
    n_pages, page, kv, d, used = 141_000, 16, 8, 128, 40
    big = [torch.empty(n_pages, page, kv, d, dtype=BF, device="cuda") for _ in range(2)]
    small = [torch.randn(used, page, kv, d, generator=g, device="cuda").to(BF) for _ in range(2)]
    for b, s in zip(big, small):
        b[n_pages - used:] = s
    table = torch.randperm(used, generator=g, device="cuda").int().view(2, 20)
    return cv, cv.PagedCache(*big, table + (n_pages - used)), cv.PagedCache(*small, table), g


@pytest.mark.parametrize("layout", ["tiles", "odd"])
def test_attention(far, layout):
    cv, big, small, g = far
    assert big.k.numel() > 2 ** 31
    lens = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 16, 128, generator=g, device="cuda").to(BF)
    outs = []
    for cache in (big, small):
        if layout == "odd":  # a channel less: rows that are no whole 16-byte pieces take the other kernel
            cache, x = cv.PagedCache(cache.k[..., :127], cache.v[..., :127], cache.page_table), q[..., :127]
        else:
            x = q
        out = torch.zeros(x.shape, dtype=BF, device="cuda")
        cv.tree_attention(x, out, cache, lens)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and bool(outs[0].abs().sum() > 0)


def test_rotation_and_compaction(far):
    cv, big, small, g = far
    x = torch.randn(2, 4, 24, 128, generator=g, device="cuda").to(BF)
    lens = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 2, 3, -1], [1, 3, -1, -1]], dtype=torch.int32, device="cuda")
    accept = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    for cache in (big, small):
        out = torch.empty(2, 4, 8, 128, dtype=BF, device="cuda")
        cv.qk_norm_rope(x[:, :, :8], x[:, :, 8:16], out, v=x[:, :, 16:], cache=cache, cache_len=lens)
        cv.cache_compact(cache, lens, path, accept)
    assert torch.equal(big.k[-40:], small.k) and torch.equal(big.v[-40:], small.v)


def test_fork(far):
    cv, big, small, g = far
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    tables = []
    for cache in (big, small):
        n = cache.k.shape[0]
        refs = torch.ones(n, dtype=torch.int32, device="cuda")
        refs[n - 1] = 0  # the only free page is the last one
        table = torch.cat([cache.page_table[:1], torch.full_like(cache.page_table[:1], -1)])
        table[0, 2] = n - 30
        pool = cv.PagedCache(cache.k, cache.v, table, held=ints(20, 0), refs=refs)
        cv.cache_fork(pool, ints(0), ints(1), ints(2 * 16 + 5))
        assert table[1].tolist()[:4] == [*table[0].tolist()[:2], n - 1, -1]
        assert torch.equal(cache.k[n - 1, :5], cache.k[n - 30, :5]) and torch.equal(cache.v[n - 1, :5], cache.v[n - 30, :5])
        tables.append(table - (n - 40))
    assert torch.equal(tables[0][:, :3], tables[1][:, :3])


def test_verification(cuda_lib):
    cv = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(1)
    n, T, V = 135, 8, 2_000_000
    probs = torch.empty(n, T, V, dtype=BF, device="cuda")
    assert probs.numel() > 2 ** 31
    probs[-1] = torch.softmax(3 * torch.randn(T, V, generator=g, device="cuda"), -1).to(BF)
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    tok, u = ints(n, T), torch.rand(n, T + 1, generator=g, device="cuda")
    tok[-1] = torch.randint(V, (T,), generator=g, device="cuda").int()
    tok[-1, 1] = int(probs[-1, 0].argmax())
    u[-1, 0] = 0
    slots = ints(n) - 1
    slots[-1] = 0
    got = []
    for p, t, x, s in ((probs, tok, u, slots), (probs[-1:].clone(), tok[-1:].clone(), u[-1:].clone(), slots[-1:].clone())):
        accept, new = ints(len(s)), ints(len(s), T)
        cv.draft_verify(p, t, x, accept, new, cache_idx=s)
        got.append((accept[-1], new[-1]))
    assert got[0][0] == got[1][0] >= 2 and torch.equal(got[0][1], got[1][1])
