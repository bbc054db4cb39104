"""What an earlier call left in shared memory reaches no output: equal bits whatever ran before."""
from __future__ import annotations

import pytest
import torch

import attn_reference as ref
from test_gpu_attention import BF, F32, check, make

pytestmark = pytest.mark.gpu


def before(cv, T, G, d, dtype, parent):
    """A call of the same kernel whose drafts see all before them, or themselves alone, in every block of the GPU."""
    n, page = 400, 16
    k = torch.zeros(n * 2, page, 1, d, dtype=dtype, device="cuda")
    cache = cv.PagedCache(k, k.clone(), torch.arange(2 * n, dtype=torch.int32, device="cuda").view(n, 2))
    q = torch.zeros(n, T, G, d, dtype=dtype, device="cuda")
    parents = torch.tensor([parent] * n, dtype=torch.int32, device="cuda")
    cv.tree_attention(q, torch.empty_like(q), cache, torch.full((n,), 9, dtype=torch.int32, device="cuda"), parent=parents)


@pytest.mark.parametrize("dtype,T,G,d", [(F32, 8, 1, 128), (F32, 8, 1, 64), (F32, 8, 1, 256), (F32, 4, 2, 128), (F32, 4, 1, 128), (F32, 16, 2, 128),
                                         (BF, 8, 1, 128), (BF, 20, 8, 128), (BF, 8, 1, 256)])
def test_equal_bits(cuda_lib, dtype, T, G, d):
    """Rows past a sequence's drafts find the masks that the call before left there: all drafts, their own place, or one late draft."""
    cv = cuda_lib
    top = T - 3 if T > 4 else T - 1
    late = [-1] * top + [top - 2 + i % 2 for i in range(T - top)]
    counts = [1 + (3 * i) % top for i in range(40)]
    for seed in range(3):
        lens = [8 * i if i < 30 else (997 * (i + 1) * (seed + 3)) % 2300 for i in range(40)]
        x = make(lens, counts, T, 2, G, d, 16, dtype, tree=True, ragged=True, seed=seed)
        outs = []
        cache = cv.PagedCache(x["k"].cuda(), x["v"].cuda(), x["table"].cuda())
        q, cu, parent = x["q"].contiguous().cuda(), x["cu"].cuda(), x["parent"].cuda()
        n, slots = torch.tensor(lens, dtype=torch.int32, device="cuda"), x["slots"].cuda()
        for earlier in (ref.chain(T), [-1] * T, late):
            out = torch.zeros_like(q)
            torch.cuda.synchronize()
            before(cv, T, G, d, dtype, earlier)
            cv.tree_attention(q, out, cache, n, parent=parent, cu_draft=cu, T=T, cache_idx=slots)
            outs.append(out)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]), seed
    check(x, outs[0].cpu(), [0] * 40)
