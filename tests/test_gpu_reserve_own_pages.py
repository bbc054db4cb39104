"""Growth with the slots' lengths: pages that are to be written and that another slot holds too are replaced by copies, against the same
calls on lists; and a fork that is rolled back and goes on."""
from __future__ import annotations

import random

import pytest
import torch

import attn_reference as ref
from test_gpu_pages import ints, make, same
from test_gpu_qk_norm_rope import angles, close
from test_gpu_shared_pages import forked, rows

pytestmark = pytest.mark.gpu


def reserve(pool, idx, n_tokens, lens):
    """Returns err and the (new page, old page, rows) to copy; counts are those before the call."""
    refs, err, copies, named, room, out, last = list(pool.refs), [], [], set(), pool.refs.count(0), False, []
    for slot, n, L in zip(idx, n_tokens, lens):
        e, shared, grow = 0, [], 0
        if slot >= 0:
            top = len(pool.table[0]) * pool.page
            if slot >= len(pool.table) or slot in named:
                e = 1
            elif not 0 <= n <= top or not 0 <= L <= pool.held[slot] * pool.page:
                e = 64
            else:
                grow = max(0, pool.pages(n) - pool.held[slot])
                held = range(L // pool.page, min(pool.held[slot], pool.pages(n)) if L < n else 0)
                if any(not 0 <= pool.table[slot][x] < len(refs) for x in held):
                    e, grow = 128, 0
                else:
                    shared = [x for x in held if refs[pool.table[slot][x]] > 1]
            named.add(slot)
            need = len(shared) + grow
            if need:
                out = out or need > room
                if out:
                    e = 1024
                else:
                    room -= need
                    for x in shared:
                        old, new = pool.table[slot][x], pool.take()
                        pool.table[slot][x] = new
                        last.append(old)
                        if x == L // pool.page and L % pool.page:
                            copies.append((new, old, L % pool.page))
                    for c in range(grow):
                        pool.table[slot][pool.held[slot] + c] = pool.take()
                    pool.held[slot] += grow
        err.append(e)
    for old in last:
        pool.refs[old] -= 1
    return err, copies


@pytest.mark.parametrize("seed", range(8))
def test_a_life_of_calls(cuda_lib, seed):
    cv, rng = cuda_lib, random.Random(seed)
    n_slots, page = 12, rng.choice([1, 4, 16])
    cache, pool = make(cv, rng, n_slots, rng.choice([25, 60, 90]), 9, page, 5, shared=0.4, d=rng.choice([8, 5]),
                       dtype=rng.choice([torch.bfloat16, torch.float32]))
    k, v = cache.k.cpu(), cache.v.cpu()
    replaced = 0
    for _ in range(40):
        n = rng.randint(1, 6)
        idx = [rng.randint(-1, n_slots - (rng.random() < 0.8)) for _ in range(n)]
        err = ints([-7] * n)
        op = rng.choice(["reserve", "reserve", "fork", "free"])
        if op == "reserve":
            lens = [rng.randint(0, pool.held[a] * page) if 0 <= a < n_slots and rng.random() < 0.9 else rng.randint(-1, 9 * page) for a in idx]
            tok = [min(max(L + rng.randint(-2, 2 * page), -1), 9 * page + 1) for L in lens]
            want, copies = reserve(pool, idx, tok, lens)
            replaced += len(copies)
            cv.cache_reserve(cache, ints(tok), cache_len=ints(lens), cache_idx=ints(idx), err=err)
        elif op == "free":
            tok, copies = [rng.randint(0, 9 * page) for _ in range(n)], []
            want = pool.free(idx, tok)
            cv.cache_free(cache, ints(tok), cache_idx=ints(idx), err=err)
        else:
            src = [rng.randint(0, n_slots - 1) for _ in range(n)]
            tok = [rng.randint(0, pool.held[a] * page) for a in src]
            want, copies = pool.fork(src, idx, tok)
            cv.cache_fork(cache, ints(src), ints(idx), ints(tok), err=err)
        for new, old, count in copies:
            k[:, new, :count], v[:, new, :count] = k[:, old, :count], v[:, old, :count]
        assert err.tolist() == want, op
        same(cache, pool)
    assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v)
    assert page == 1 or replaced > 0


@pytest.mark.parametrize("every", [1, 3000, 6400])
def test_pages_from_far_apart(cuda_lib, every):
    """Eleven shared pages of one slot and one of another, replaced by free pages of one or several passes over the counts."""
    cv, n_pages, page = cuda_lib, 110_000, 4
    refs = torch.ones(n_pages, dtype=torch.int32)
    refs[torch.arange(20_000, n_pages, every)] = 0
    refs[:12] = 2
    table = [list(range(12)) + [-1] * 3, list(range(11, -1, -1)) + [-1] * 3]
    k = torch.randn(n_pages, page, 1, 4, generator=torch.Generator().manual_seed(0))
    cache = cv.PagedCache(k.cuda(), -k.cuda(), ints(table), held=ints([12, 12]), refs=refs.cuda())
    pool = ref.Pool(table, [12, 12], refs.tolist(), page)
    err = ints([-7, -7])
    tok, lens = [55, 46], [6, 45]
    want, copies = reserve(pool, [0, 1], tok, lens)
    assert len(copies) == 2
    cv.cache_reserve(cache, ints(tok), cache_len=ints(lens), err=err)
    assert err.tolist() == want == [0, 0]
    same(cache, pool)
    for new, old, count in copies:
        k[new, :count] = k[old, :count]
    assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), -k)


@pytest.mark.parametrize("d", [64, 20])
@pytest.mark.parametrize("side", [0, 1])
def test_a_rolled_back_fork_goes_on(cuda_lib, d, side):
    """Forked at 32, trimmed to 20 and grown to 34 tokens: the other side keeps its bits, and this one has its own 20 and 14 new tokens."""
    cv = cuda_lib
    cache = forked(cv, d)
    other, mine = rows(cache, 1 - side, 32).clone(), rows(cache, side, 20).clone()
    cv.cache_free(cache, ints([20]), cache_idx=ints([side]))
    cv.cache_reserve(cache, ints([34]), cache_len=ints([20]), cache_idx=ints([side]))
    q, k = torch.randn(1, 14, 4, d, device="cuda"), torch.randn(1, 14, 2, d, device="cuda")
    v, out, err = torch.randn_like(k), torch.empty_like(q), ints([-7])
    cs = angles(40, d)
    for layer in range(2):
        cv.qk_norm_rope(q, k, out, v=v, cos_sin=cs.cuda(), cache=cache.layer(layer), cache_len=ints([20]), cache_idx=ints([side]), err=err)
        assert err.tolist() == [0]
    assert torch.equal(rows(cache, 1 - side, 32), other)
    now = rows(cache, side, 34)
    assert torch.equal(now[:, :, :20], mine)
    z = cs[20:34]
    want = ref.norm_rope(k.cpu()[0], None, z[:, :d // 2], z[:, d // 2:], False, True, 1e-6)
    for layer in range(2):
        assert close(now[0, layer, 20:].cpu(), want, k, None, torch.float32) and torch.equal(now[1, layer, 20:], v[0])
    assert int(cache.refs.sum()) == int(cache.held.sum()) and int(cache.refs.min()) == 0


def test_both_sides_at_once(cuda_lib):
    """Each gets a copy, and the page that both held is free."""
    cv = cuda_lib
    cache = forked(cv)
    sides = [rows(cache, s, 20).clone() for s in (0, 1)]
    cv.cache_free(cache, ints([20, 20]), cache_idx=ints([0, 1]))
    cv.cache_reserve(cache, ints([21, 40]), cache_len=ints([20, 20]), cache_idx=ints([0, 1]))
    assert cache.page_table[:2, :3].tolist() == [[0, 2, -1], [0, 3, 4]]
    assert cache.refs.tolist() == [2, 0, 1, 1, 1] + [0] * 7 and cache.held.tolist() == [2, 3, 0]
    for s in (0, 1):
        assert torch.equal(rows(cache, s, 20), sides[s])


def test_captured(cuda_lib):
    """A replay finds the pages of its time."""
    cv = cuda_lib
    cache = forked(cv)
    mine, want, lens, side = rows(cache, 1, 20).clone(), ints([33]), ints([32]), ints([1])
    cv.cache_reserve(cache, want, cache_len=lens, cache_idx=side)
    assert cache.page_table[1].tolist()[:3] == [0, 1, 3]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cv.cache_reserve(cache, want, cache_len=lens, cache_idx=side)
    graph.replay()
    assert cache.page_table[1].tolist()[:3] == [0, 1, 3]
    lens.fill_(20)
    graph.replay()
    graph.replay()
    assert cache.page_table[1].tolist()[:3] == [0, 4, 3] and cache.refs.tolist()[:6] == [2, 1, 1, 1, 1, 0]
    assert torch.equal(rows(cache, 1, 20), mine)
