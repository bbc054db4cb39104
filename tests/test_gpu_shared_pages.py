"""Pages that more than one slot holds are not written: a fork that is rolled back into them and goes on leaves the other side's bits."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
SHARED = 4096


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def forked(cv, d=64, layers=2, counts=True, page=16):
    """Slot 0 with 40 tokens, slot 1 forked from its first 32; the pages past them are spare."""
    g = torch.Generator(device="cuda").manual_seed(d)
    shape = (layers, 12, page, 2, d)
    k, v = (torch.randn(shape, generator=g, device="cuda") for _ in range(2))
    cache = cv.PagedCache(k, v, torch.full((3, 6), -1, dtype=torch.int32, device="cuda"), held=ints(0, 0, 0), refs=ints(*[0] * 12))
    cv.cache_reserve(cache, ints(40))
    cv.cache_fork(cache, ints(0), ints(1), ints(32))
    assert cache.page_table[:2, :3].tolist() == [[0, 1, 2], [0, 1, -1]] and cache.refs.tolist()[:4] == [2, 2, 1, 0]
    return cache


def rows(cache, slot, n):
    at = torch.arange(n, device="cuda")
    pages = cache.page_table[slot].long()[at // 16]
    return torch.stack([cache.k[:, pages, at % 16], cache.v[:, pages, at % 16]])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("d", [64, 20])
def test_a_rolled_back_fork_goes_on(cuda_lib, d, side, packed):
    """Either side is trimmed to 20 tokens, and 14 more are written: 12 of them would stand in the page of both."""
    cv = cuda_lib
    cache = forked(cv, d)
    other, mine, whole = rows(cache, 1 - side, 32).clone(), rows(cache, side, 20).clone(), cache.k.clone()
    cv.cache_free(cache, ints(20), cache_idx=ints(side))
    cv.cache_reserve(cache, ints(34), cache_idx=ints(side))
    q, k = torch.randn(1, 14, 4, d, device="cuda"), torch.randn(1, 14, 2, d, device="cuda")
    out, err, kw = torch.full_like(q, 7.0), ints(-7), {}
    if packed:
        q, k, out, kw = q[0], k[0], out[0], dict(cu_seqlens=ints(0, 14), max_seqlen=14)
    one = cache.layer(0)
    cv.qk_norm_rope(q, k, out, v=k.clone(), cache=one, cache_len=ints(20), cache_idx=ints(side), err=err, **kw)
    assert torch.equal(rows(cache, 1 - side, 32), other) and torch.equal(rows(cache, side, 20), mine)
    assert err.tolist() == [SHARED]
    left = (out == 7).flatten(-2).all(-1).flatten().tolist()
    assert left == [True] * 12 + [False] * 2  # the last two have a page of their own
    page = int(cache.page_table[side, 2])
    whole[0, page, :2] = cache.k[0, page, :2]
    assert torch.equal(cache.k, whole) and not torch.equal(cache.k[0, page, 0], cache.v[0, page, 0] + 1)
    # a handle without counts is told nothing of the sharing
    cv.qk_norm_rope(q, k, out, v=k.clone(), cache=cv.PagedCache(one.k, one.v, one.page_table), cache_len=ints(20), cache_idx=ints(side), err=err, **kw)
    assert err.tolist() == [0] and not bool((out == 7).any())


@pytest.mark.parametrize("side", [0, 1])
def test_compaction_into_a_shared_page(cuda_lib, side):
    """A path that would move rows into it is flagged; one whose rows stay there, or move behind it, is not."""
    cv = cuda_lib
    cache = forked(cv)
    cv.cache_free(cache, ints(20), cache_idx=ints(side))
    cv.cache_reserve(cache, ints(36), cache_idx=ints(side))
    k, v = cache.k.clone(), cache.v.clone()
    err, new = ints(-7), ints(-3)
    path = torch.full((1, 16), -1, dtype=torch.int32, device="cuda")
    path[0, :3] = ints(0, 2, 13)
    cv.cache_compact(cache, ints(20), path, ints(3), new_len=new, cache_idx=ints(side), err=err)
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)
    assert err.tolist() == [SHARED] and new.tolist() == [-3]
    cv.cache_compact(cache, ints(20), path, ints(1), new_len=new, cache_idx=ints(side), err=err)
    assert err.tolist() == [0] and new.tolist() == [21] and torch.equal(cache.k, k)
    path[0, :2] = ints(0, 3)
    cv.cache_compact(cache, ints(31), path, ints(2), new_len=new, cache_idx=ints(side), err=err)
    own = int(cache.page_table[side, 2])
    k[:, own, 0], v[:, own, 0] = k[:, own, 2].clone(), v[:, own, 2].clone()
    assert err.tolist() == [0] and new.tolist() == [33] and torch.equal(cache.k, k) and torch.equal(cache.v, v)
