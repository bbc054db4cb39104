"""Packed rows whose counts fall, leave the rows or belong to empty sequences: each sequence is judged by its own counts, as attention
judges it, and every good one's keys and values are written."""
from __future__ import annotations

import pytest
import torch

import attn_reference as ref
from test_gpu_qk_norm_rope import angles, close

pytestmark = pytest.mark.gpu
F32 = torch.float32
#     counts, longest, rows, slots, lengths, flags (slots n_slots and up are none; pages hold 24 tokens a slot)
CASES = [
    ([0, 4, 3, 7], 4, 7, [0, 1, 2], [0, 0, 0], [0, 16, 0]),
    ([0, 4, 3, 12], 9, 12, [0, 1, 2], [3, 0, 5], [0, 16, 0]),
    ([0, 4, 3, 12], 4, 12, [0, 1, 2], [3, 0, 5], [0, 16, 16]),
    ([2, 9, 1], 9, 10, [0, 1], [0, 0], [0, 16]),
    ([5, 9, 0, 4], 4, 9, [2, 1, 0], [1, 0, 2], [0, 16, 0]),
    ([0, 6, 0, 6, 2, 6], 6, 6, [0, 1, 2, 3, -1], [0, 0, 1, 0, 0], [0, 16, 0, 16, 0]),
    ([0, 3, 3, 5], 4, 5, [0, 4, 2], [0, 0, 0], [0, 1, 0]),          # an empty sequence of no slot
    ([0, 3, 3, 5], 4, 5, [0, 1, 2], [0, -1, 0], [0, 64, 0]),        # ... of no length
    ([0, 3, 3, 5], 4, 5, [0, -1, 2], [0, -1, 0], [0, 0, 0]),        # ... padded
    ([-2, 3, 5, 11], 8, 10, [0, 1, 2], [0, 0, 0], [16, 0, 16]),     # rows that are not there
    ([0, 5, 5], 4, 3, [0, 1], [0, 0], [16, 16]),
    ([0, 2, 4], 2, 4, [0, 1], [23, 22], [64, 0]),
]


def inputs(cu, total, d, kv=2, H=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(total, h, d, generator=g) for h in (H, kv, kv))
    n = len(cu) - 1
    return q, k, v, torch.randperm(4 * 3, generator=g).int().view(4, 3), n


@pytest.mark.parametrize("d", [64, 20])  # rows of 16-byte pieces, and the other kernel
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cu,T,total,slots,lens,flags", CASES)
def test_counts(cuda_lib, cu, T, total, slots, lens, flags, in_place, d):
    cv = cuda_lib
    q, k, v, table, n = inputs(cu, total, d)
    page, cs = 8, angles(40, d)
    cache = cv.PagedCache(*(torch.full((12, page, 2, d), 7.0, device="cuda") for _ in range(2)), table.cuda())
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    a, b = q.cuda(), k.cuda()
    out, k_out = (a, b) if in_place else (torch.full_like(a, 7.0), torch.full_like(b, 7.0))
    err = ints([-7] * n)
    cv.qk_norm_rope(a, b, out, k_out=k_out, v=v.cuda(), cos_sin=cs.cuda(), cache=cache, cache_len=ints(lens), cu_seqlens=ints(cu),
                    max_seqlen=T, cache_idx=ints(slots), err=err)
    torch.cuda.synchronize()
    assert err.tolist() == flags
    want_q, want_k = (q, k) if in_place else (torch.full_like(q, 7.0), torch.full_like(k, 7.0))
    want_q, want_k = want_q.double(), want_k.double()
    touched = torch.zeros(12, page, dtype=torch.bool)
    for s in range(n):  # a row's last owner has it in the outputs
        if flags[s] or slots[s] < 0 or cu[s + 1] <= cu[s]:
            continue
        rows = slice(cu[s], cu[s + 1])
        pos = lens[s] + torch.arange(cu[s + 1] - cu[s])
        turned = [ref.norm_rope(x[rows], None, cs[pos][:, :d // 2], cs[pos][:, d // 2:], False, True, 1e-6) for x in (q, k)]
        want_q[rows], want_k[rows] = turned
        pg = table[slots[s], pos // page].long()
        assert close(cache.k[pg, pos % page].cpu(), turned[1], k, None, F32)
        assert torch.equal(cache.v[pg, pos % page].cpu(), v[rows])
        touched[pg, pos % page] = True
    assert close(out.cpu(), want_q, q, None, F32) and close(k_out.cpu(), want_k, k, None, F32)
    assert bool((cache.k.cpu()[~touched] == 7).all()) and bool((cache.v.cpu()[~touched] == 7).all())


@pytest.mark.parametrize("cu,T,total,slots,lens,flags", CASES)
def test_the_same_flags_as_attention(cuda_lib, cu, T, total, slots, lens, flags):
    cv = cuda_lib
    q, k, v, table, n = inputs(cu, total, 64)
    cache = cv.PagedCache(*(torch.zeros(12, 8, 2, 64, device="cuda") for _ in range(2)), table.cuda())
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    err = ints([-7] * n)
    q = torch.zeros(total, 4, 64, device="cuda")
    cv.tree_attention(q, torch.empty_like(q), cache, ints(lens), cu_draft=ints(cu), T=T, cache_idx=ints(slots), err=err)
    assert err.tolist() == flags


def test_more_sequences_than_threads_and_no_cache(cuda_lib):
    """700 sequences, every seventh one's counts fall by one row; without a cache the last owner of a row decides its position."""
    cv = cuda_lib
    cu = [0]
    for s in range(700):
        cu.append(cu[-1] - 1 if s % 7 == 6 else cu[-1] + s % 3)
    total = max(cu)
    q = torch.randn(total, 1, 32, generator=torch.Generator().manual_seed(1))
    out, err = torch.full_like(q, 7.0).cuda(), torch.full((700,), -7, dtype=torch.int32, device="cuda")
    cs = angles(4, 32)
    cv.qk_norm_rope(q.cuda(), None, out, cos_sin=cs.cuda(), cache_len=torch.ones(700, dtype=torch.int32, device="cuda"),
                    cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen=2, err=err)
    assert err.tolist() == [16 if s % 7 == 6 else 0 for s in range(700)]
    want = torch.full_like(q, 7.0).double()
    for s in range(700):
        if cu[s + 1] > cu[s]:
            z = cs[1 + torch.arange(cu[s + 1] - cu[s])]
            want[cu[s]:cu[s + 1]] = ref.norm_rope(q[cu[s]:cu[s + 1]], None, z[:, :16], z[:, 16:], False, True, 1e-6)
    assert close(out.cpu(), want, q, None, F32)
