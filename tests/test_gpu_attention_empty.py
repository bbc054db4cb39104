"""Calls without a token: their sequences' flags are this call's, as those of the verification are."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
#     counts, slots (4 there are), lengths (tables of 24 tokens), flags
CASES = [([0, 0, 0, 0], [0, 1, 2], [0, 5, 24], [0, 0, 0]), ([0, 0, 0, 0], [0, 4, -1], [-1, 0, -1], [64, 1, 0]), ([0, 5, 0, 0], [0, 1, 2], [0, 0, 25], [16, 16, 64]),
         ([0, -1, 0, 3], [0, -1, 2], [0, 0, 0], [16, 0, 16])]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def old():
    return ints([-7] * 3)


def paged(cv, dtype=torch.bfloat16, d=64):
    k = torch.zeros(12, 8, 2, d, dtype=dtype, device="cuda")
    return cv.PagedCache(k, torch.zeros_like(k), torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 20])
@pytest.mark.parametrize("cu,slots,lens,flags", CASES)
def test_no_packed_rows(cuda_lib, cu, slots, lens, flags, d, dtype):
    cv = cuda_lib
    cache, q, k = paged(cv, dtype, d), torch.empty(0, 4, d, dtype=dtype, device="cuda"), torch.empty(0, 2, d, dtype=dtype, device="cuda")
    err = old()
    cv.tree_attention(q, torch.empty_like(q), cache, ints(lens), cu_draft=ints(cu), T=4, cache_idx=ints(slots), err=err)
    assert err.tolist() == flags
    err = old()
    cv.qk_norm_rope(q, k, torch.empty_like(q), cache=cache, cache_len=ints(lens), cu_seqlens=ints(cu), max_seqlen=4, cache_idx=ints(slots),
                    err=err)
    assert err.tolist() == flags
    cv.tree_attention(q, torch.empty_like(q), cache, ints(lens), cu_draft=ints(cu), T=4, cache_idx=ints(slots))
    cv.qk_norm_rope(q, k, torch.empty_like(q), cache=cache, cache_len=ints(lens), cu_seqlens=ints(cu), max_seqlen=4, cache_idx=ints(slots))
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 20])
def test_no_tokens_a_sequence(cuda_lib, d):
    cv = cuda_lib
    cache, q, k = paged(cv, d=d), torch.empty(3, 0, 4, d, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 0, 2, d, dtype=torch.bfloat16, device="cuda")
    err = old()
    cv.qk_norm_rope(q, k, torch.empty_like(q), cache=cache, cache_len=ints([0, 25, 24]), cache_idx=ints([4, 1, 2]), err=err)
    assert err.tolist() == [1, 64, 0]
    # packed rows of sequences that may hold none
    q, k = torch.full((6, 4, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((6, 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    err = old()
    cv.qk_norm_rope(q, k, q, k_out=k, cache=cache, cache_len=ints([0, 0, 0]), cu_seqlens=ints([0, 3, 3, 6]), max_seqlen=0, err=err)
    assert err.tolist() == [16, 0, 16] and bool((q == 7).all()) and bool((k == 7).all()) and bool((cache.k == 0).all())


def test_no_heads(cuda_lib):
    cv = cuda_lib
    q = torch.empty(3, 2, 0, 64, device="cuda")
    err = old()
    cv.qk_norm_rope(q, None, torch.empty_like(q), cache_len=ints([0, -1, 3]), err=err)
    assert err.tolist() == [0, 64, 0]


def test_in_a_graph(cuda_lib):
    """A captured call without rows raises the flags of the counts that it finds."""
    cv = cuda_lib
    cache, q, k = paged(cv), torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu, lens, errs = ints([0, 0, 0, 0]), ints([0, 0, 0]), [old(), old()]

    def calls():
        cv.tree_attention(q, q.clone(), cache, lens, cu_draft=cu, T=4, err=errs[0])
        cv.qk_norm_rope(q, k, q.clone(), cache=cache, cache_len=lens, cu_seqlens=cu, max_seqlen=4, err=errs[1])

    calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    cu.copy_(ints([0, 2, 1, 1]))
    for flags in ([16, 16, 16], [16, 16, 16]):
        for e in errs:
            e.fill_(-7)
        graph.replay()
        assert errs[0].tolist() == errs[1].tolist() == flags
    cu.zero_()
    graph.replay()
    assert errs[0].tolist() == errs[1].tolist() == [0, 0, 0]
