"""The pages of a cache against the same calls on lists: equal tables, counts and bits."""
from __future__ import annotations

import random

import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(cv, rng, n_slots, n_pages, max_pages, page, used, layers=2, n_kv=2, d=8, dtype=torch.bfloat16, shared=0):
    """A pool whose first `used` slots hold random pages, some of them shared."""
    order = list(range(n_pages))
    rng.shuffle(order)
    table = [[-9] * max_pages for _ in range(n_slots)]
    held, refs = [0] * n_slots, [0] * n_pages
    for s in range(used):
        h = min(rng.randint(0, max_pages), len(order))
        for c in range(h):
            table[s][c] = order.pop() if not (shared and s and rng.random() < shared and held[s - 1] > c) else table[s - 1][c]
            refs[table[s][c]] += 1
        held[s] = h
    g = torch.Generator().manual_seed(rng.randrange(1 << 30))
    shape = (layers, n_pages, page, n_kv, d)
    k, v = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
    cache = cv.PagedCache(k, v, ints(table), held=ints(held), refs=ints(refs))
    return cache, ref.Pool(table, held, refs, page)


def same(cache, pool):
    assert cache.held.tolist() == pool.held
    assert cache.refs.tolist() == pool.refs
    assert cache.page_table.tolist() == pool.table


@pytest.mark.parametrize("seed", range(6))
def test_a_life_of_calls(cuda_lib, seed):
    """Random reserves, forks and frees, with slots, lengths and pages that are not there among them."""
    cv, rng = cuda_lib, random.Random(seed)
    n_slots, page = 12, rng.choice([1, 4, 16])
    cache, pool = make(cv, rng, n_slots, rng.choice([30, 90]), 9, page, 5)
    k, v = cache.k.cpu(), cache.v.cpu()
    for _ in range(25):
        n = rng.randint(1, 6)
        idx = [rng.randint(-1, n_slots) for _ in range(n)]
        tok = [rng.randint(-1, 9 * page + 1) for _ in range(n)]
        err = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        op = rng.choice(["reserve", "fork", "free"])
        if op == "reserve":
            want = pool.reserve(idx, tok)
            cv.cache_reserve(cache, ints(tok), cache_idx=ints(idx), err=err)
        elif op == "free":
            want = pool.free(idx, tok)
            cv.cache_free(cache, ints(tok), cache_idx=ints(idx), err=err)
        else:
            src = [rng.randint(-1, n_slots) for _ in range(n)]
            tok = [rng.randint(0, pool.held[a] * page) if 0 <= a < n_slots and rng.random() < 0.8 else t for a, t in zip(src, tok)]
            want, copies = pool.fork(src, idx, tok)
            for new, old, rows in copies:
                k[:, new, :rows], v[:, new, :rows] = k[:, old, :rows], v[:, old, :rows]
            cv.cache_fork(cache, ints(src), ints(idx), ints(tok), err=err)
        assert err.tolist() == want, op
        same(cache, pool)
    assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v)


@pytest.mark.parametrize("n_pages", [1, 15, 16, 17, 16384, 16385, 70001])
def test_pages_are_given_in_order(cuda_lib, n_pages):
    cv, rng = cuda_lib, random.Random(n_pages)
    table = torch.full((5, n_pages), -9, dtype=torch.int32, device="cuda")
    refs = torch.tensor([rng.random() < 0.6 for _ in range(n_pages)], device="cuda").int()
    free = (refs == 0).nonzero().flatten().tolist()
    kv = torch.zeros(n_pages, 2, 1, 8, device="cuda")
    cache = cv.PagedCache(kv, kv.clone(), table, held=ints([0] * 5), refs=refs)
    want = [len(free) // 3, 0, len(free) // 2, 1, 10 ** 6 if n_pages > 10 ** 6 else len(free)]
    err = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    cv.cache_reserve(cache, ints([min(2 * w, 2 * n_pages) for w in want]), err=err)
    at, out = 0, False
    for s, w in enumerate(want):
        out = out or at + w > len(free)
        if w and out:
            assert err[s] == 1024 and cache.held[s] == 0 and bool((table[s] == -9).all())
            continue
        assert err[s] == 0 and table[s, :w].tolist() == free[at:at + w] and bool((table[s, w:] == -9).all())
        at += w
    assert int((refs == 0).sum()) == len(free) - at


def test_two_sequences_name_a_slot(cuda_lib):
    cv = cuda_lib
    cache, pool = make(cv, random.Random(1), 6, 40, 6, 4, 3)
    for call, want in ((cv.cache_reserve, pool.reserve), (cv.cache_free, pool.free)):
        err = ints([-7] * 5)
        call(cache, ints([24, 3, 24, 9, 1]), cache_idx=ints([4, 5, 4, 5, 4]), err=err)
        assert err.tolist() == want([4, 5, 4, 5, 4], [24, 3, 24, 9, 1]) == [0, 0, 1, 1, 1]
        same(cache, pool)


def test_more_sequences_than_threads(cuda_lib):
    cv, rng = cuda_lib, random.Random(5)
    n = 2500
    cache, pool = make(cv, rng, n, 6000, 4, 2, 300, layers=1, n_kv=1)
    tok = [rng.randint(0, 8) for _ in range(n)]
    err = ints([-7] * n)
    cv.cache_reserve(cache, ints(tok), err=err)
    assert err.tolist() == pool.reserve(range(n), tok)
    same(cache, pool)
    keep = [rng.randint(0, 8) for _ in range(n)]
    idx = list(range(n))
    rng.shuffle(idx)
    cv.cache_free(cache, ints(keep), cache_idx=ints(idx), err=err)
    assert err.tolist() == pool.free(idx, keep)
    same(cache, pool)
    cv.cache_free(cache)
    pool.free(range(n), [0] * n)
    same(cache, pool)
    assert sum(pool.refs) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [128, 8, 5, 1])
@pytest.mark.parametrize("layers", [1, 3])
def test_fork_copies_the_last_page(cuda_lib, d, layers, dtype):
    cv, rng = cuda_lib, random.Random(d)
    cache, pool = make(cv, rng, 10, 60, 5, 16, 4, layers=layers, n_kv=3, d=d, dtype=dtype, shared=0.3)
    k, v = cache.k.cpu(), cache.v.cpu()
    src = [0, 1, 2, 3, 1]
    tok = [rng.randint(0, 16 * pool.held[a]) for a in src]
    want, copies = pool.fork(src, [4, 5, 6, 7, 8], tok)
    cv.cache_fork(cache, ints(src), ints([4, 5, 6, 7, 8]), ints(tok))
    for new, old, rows in copies:
        k[:, new, :rows], v[:, new, :rows] = k[:, old, :rows], v[:, old, :rows]
    same(cache, pool)
    assert want == [0] * 5 and torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v)


def test_a_page_that_is_not_there(cuda_lib):
    """Fork and free look at every page first and leave the slot as it was."""
    cv = cuda_lib
    cache, pool = make(cv, random.Random(3), 6, 40, 6, 4, 0)
    pool.reserve([0, 1], [22, 9])
    cv.cache_reserve(cache, ints([22, 9]), cache_idx=ints([0, 1]))
    cache.page_table[0, 2] = 40
    pool.table[0][2] = 40
    before = cache.refs.clone()
    err = ints([-7, -7])
    cv.cache_fork(cache, ints([0, 1]), ints([2, 3]), ints([21, 9]), err=err)
    want, _ = pool.fork([1], [3], [9])
    assert err.tolist() == [128, 0] and cache.held.tolist()[:4] == [6, 3, 0, 3]
    assert bool((cache.page_table[2, 0:5] == -9).all())
    assert int(cache.refs.sum()) == int(before.sum()) + 3
    err = ints([-7])
    cv.cache_free(cache, cache_idx=ints([0]), err=err)
    assert err.tolist() == [128] and cache.held[0] == 6 and cache.page_table[0].tolist() == pool.table[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,page,layers", [(128, 16, 2), (8, 3, 1), (5, 4, 3), (1, 1, 1), (64, 256, 1)])
@pytest.mark.parametrize("T", [1, 4, 31, 128])
def test_compact(cuda_lib, T, d, page, layers, dtype):
    cv, rng = cuda_lib, random.Random(T * d)
    n = 7
    lens = [rng.choice([0, 1, page, 2 * page + 1, 77]) for _ in range(n)]
    per = [-(-(L + T) // page) for L in lens]
    order = list(range(sum(per) + 2))
    rng.shuffle(order)
    table = [[order.pop() for _ in range(p)] + [10 ** 9] * (max(per) - p) for p in per]
    slots = list(range(n))
    rng.shuffle(slots)
    rows = [None] * n
    for s, slot in enumerate(slots):
        rows[slot] = table[s]
    slots[2] = -1
    g = torch.Generator().manual_seed(T)
    k, v = (torch.randn(layers, sum(per) + 2, page, 2, d, generator=g).to(dtype) for _ in range(2))
    accept = [rng.randint(0, T) for _ in range(n)]
    accept[0], accept[1] = T, 1
    path = torch.full((n, T), -1, dtype=torch.int32)
    for s in range(n):
        path[s, :accept[s]] = torch.tensor(sorted(rng.sample(range(T), accept[s])), dtype=torch.int32)
    cache = cv.PagedCache(k.cuda(), v.cuda(), ints(rows))
    new_len, err = ints([-3] * n), ints([-7] * n)
    cv.cache_compact(cache, ints(lens), path.cuda(), ints(accept), new_len=new_len, cache_idx=ints(slots), err=err)
    torch.cuda.synchronize()
    want_k, want_v = k.clone(), v.clone()
    for s in range(n):
        if slots[s] < 0:
            continue
        for i in range(accept[s]):
            a, b = lens[s] + int(path[s, i]), lens[s] + i
            for w, x in ((want_k, k), (want_v, v)):
                w[:, table[s][b // page], b % page] = x[:, table[s][a // page], a % page]
    assert err.tolist() == [0] * n
    assert new_len.tolist() == [lens[s] + accept[s] if slots[s] >= 0 else -3 for s in range(n)]
    assert torch.equal(cache.k.cpu(), want_k) and torch.equal(cache.v.cpu(), want_v)


def test_compact_flags(cuda_lib):
    cv = cuda_lib
    n, T, page = 8, 4, 4
    table = torch.arange(n * 3, dtype=torch.int32).view(n, 3)
    table[5, 1] = -2
    k = torch.randn(1, n * 3, page, 1, 8).cuda()
    cache = cv.PagedCache(k, k.clone(), table.cuda())
    path = torch.tensor([[0, 2, 3, -1]] * n, dtype=torch.int32)
    path[2], path[3] = torch.tensor([0, 2, 2, 3]), torch.tensor([0, 2, 4, -1])
    lens = [0, 0, 0, 0, -1, 3, 10, 0]
    err, new_len = ints([-7] * n), ints([-3] * n)
    cv.cache_compact(cache, ints(lens), path.cuda(), ints([3, 5, 3, 3, 3, 3, 3, 3]), new_len=new_len,
                     cache_idx=ints([0, 1, 2, 3, 4, 5, 6, n]), err=err)
    assert err.tolist() == [0, 4, 32, 32, 64, 128, 64, 1]
    assert new_len.tolist() == [3] + [-3] * 7
    assert torch.equal(cache.k[:, 3:], cache.v[:, 3:])
