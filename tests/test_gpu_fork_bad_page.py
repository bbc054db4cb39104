"""Forks whose source holds a page that is not there: nothing of them is done, and the pages go to the others."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(cv, table, held, refs, page=4):
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(2, len(refs), page, 1, 8, generator=g, device="cuda") for _ in range(2))
    return cv.PagedCache(k, v, ints(table), held=ints(held), refs=ints(refs))


@pytest.mark.parametrize("bad", [-1, 6, 10 ** 9])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_the_slot_is_left_as_it_was(cuda_lib, at, bad):
    """One free page, a bad fork first and a good one second."""
    cv = cuda_lib
    table = [[0, 1, 2], [3, 4, -8], [-9, -8, -7], [-6, -5, -4]]
    table[0][at] = bad
    cache = pool(cv, table, [3, 2, 0, 0], [1, 1, 1, 1, 1, 0])
    k, err = cache.k.clone(), ints([-7, -7])
    cv.cache_fork(cache, ints([0, 1]), ints([2, 3]), ints([10, 7]), err=err)
    assert err.tolist() == [128, 0]
    assert cache.page_table.tolist() == table[:3] + [[3, 5, -4]]
    assert cache.held.tolist() == [3, 2, 0, 2] and cache.refs.tolist() == [1, 1, 1, 2, 1, 1]
    k[:, 5, :3] = k[:, 4, :3]
    assert torch.equal(cache.k, k)


def test_pages_past_the_fork_are_not_looked_at(cuda_lib):
    cv = cuda_lib
    cache = pool(cv, [[0, 77, 99], [-1, -1, -1], [-1, -1, -1]], [3, 0, 0], [1, 0, 0])
    err = ints([-7, -7])
    cv.cache_fork(cache, ints([0, 0]), ints([1, 2]), ints([4, 0]), err=err)
    assert err.tolist() == [0, 0] and cache.held.tolist() == [3, 1, 0] and cache.refs.tolist() == [2, 0, 0]
    assert cache.page_table.tolist() == [[0, 77, 99], [0, -1, -1], [-1, -1, -1]]


@pytest.mark.parametrize("n_src,pages", [(1, 1), (1, 2000), (40, 300), (1500, 5)])
def test_many_and_long_sources(cuda_lib, n_src, pages):
    """Every third source has one bad page, anywhere; each is forked to a slot of its own."""
    cv = cuda_lib
    g = torch.Generator().manual_seed(pages)
    n_pages = n_src * pages + n_src + 5
    order = torch.randperm(n_pages, generator=g).int()
    table = torch.full((2 * n_src, pages + 1), -3, dtype=torch.int32)
    table[:n_src, :pages] = order[:n_src * pages].view(n_src, pages)
    held = [pages] * n_src + [0] * n_src
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[order[:n_src * pages].long()] = 1
    n_tok = torch.randint(max(1, 4 * pages - 600), 4 * pages + 1, (n_src,), generator=g).tolist()
    bad = [s for s in range(n_src) if s % 3 == 0]
    for s in bad:
        table[s, int(torch.randint(-(-n_tok[s] // 4), (1,), generator=g))] = n_pages if s % 2 else -1
    cache = pool(cv, table.tolist(), held, refs.tolist())
    before, err = cache.k.cpu(), ints([-7] * n_src)
    cv.cache_fork(cache, ints(list(range(n_src))), ints(list(range(n_src, 2 * n_src))), ints(n_tok), err=err)
    free = [int(x) for x in torch.nonzero(refs == 0).flatten()]
    want_refs, want_table, k = refs.clone(), table.clone(), before.clone()
    for s in range(n_src):
        if s in bad:
            continue
        full, rest = divmod(n_tok[s], 4)
        want_table[n_src + s, :full] = table[s, :full]
        want_refs[table[s, :full].long()] += 1
        held[n_src + s] = full + (rest > 0)
        if rest:
            new = free.pop(0)
            want_table[n_src + s, full], want_refs[new] = new, 1
            k[:, new, :rest] = before[:, int(table[s, full]), :rest]
    assert err.tolist() == [128 if s in bad else 0 for s in range(n_src)]
    assert torch.equal(cache.page_table.cpu(), want_table) and torch.equal(cache.refs.cpu(), want_refs)
    assert cache.held.tolist() == held and torch.equal(cache.k.cpu(), k)
