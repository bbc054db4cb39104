"""Tree attention of up to 8 rows a kv head over rows of whole 16-byte pieces in fp32 products (fp32, and bf16 over pages of 5
tokens), against the softmax in 64 bits."""
from __future__ import annotations

import pytest
import torch

import test_gpu_attention as base

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LENS = [0, 1, 7, 8, 9, 63, 64, 65, 300, 517]


@pytest.mark.parametrize("dtype,page", [(F32, 16), (BF, 5), (F32, 1)])
@pytest.mark.parametrize("d", [64, 48, 128, 112, 256, 200])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 8), (2, 4), (8, 1), (5, 1), (1, 3)])
def test_rows_and_heads(cuda_lib, T, G, d, dtype, page):
    x = base.make(LENS, [T] * len(LENS), T, 2, G, d, page, dtype, tree=T > 1, seed=d + T, pad=(2,))
    base.check(x, *base.call(cuda_lib, x))


@pytest.mark.parametrize("dtype,page", [(F32, 32), (BF, 5)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_ragged_drafts(cuda_lib, d, dtype, page):
    counts = [1, 4, 0, 2, 3, 1, 4, 0, 4, 2]
    x = base.make(LENS, counts, 4, 2, 2, d, page, dtype, tree="forest", ragged=True, seed=d)
    base.check(x, *base.call(cuda_lib, x))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [1.0, 4.0])
def test_maxima_that_move(cuda_lib, d, scale):
    """Scores of +-16 sqrt(d) and more: each new maximum moves the sums by far more than 2^8."""
    x = base.make([40, 3000, 701], [2] * 3, 2, 2, 4, d, 16, F32, seed=d)
    base.check(x, *base.call(cuda_lib, x, scale=scale), scale=scale)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_draft_that_is_not_finite_reaches_those_that_see_it(cuda_lib, d, bad):
    cv, T, L = cuda_lib, 4, 61
    x = base.make([L], [T], T, 1, 2, d, 16, F32, seed=7)
    x["parent"] = torch.tensor([[-1, 0, 0, 2]], dtype=torch.int32)
    x["parents"] = [[-1, 0, 0, 2]]
    clean, _ = base.call(cv, x)
    at = L + 1  # draft 1, which itself alone sees
    x["v"][int(x["table"][int(x["slots"][0]), at // 16]), at % 16, 0, 3] = bad
    got, err = base.call(cv, x)
    assert err == [0]
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[0, 1, :, 3] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert bool((torch.isnan(got[hit]) if bad != bad else got[hit] == bad).all())


@pytest.mark.parametrize("shape", [(96, 1500, 8, 8, 128, 1), (96, 1500, 32, 4, 128, 1), (64, 1500, 16, 8, 64, 4), (48, 1500, 8, 4, 256, 2),
                                   (300, 90, 8, 8, 128, 1)], ids=str)
def test_every_key_counts_once(cuda_lib, shape):
    """Queries of zero and values of one give one: sums of whole numbers, one division and one product (2^-23), and powers of two
    that are one but for 2^-22.  A key left out of 1505 would be 2^-11."""
    cv, (n, ctx, H, kv, d, T) = cuda_lib, shape
    lens = [ctx - i * 41 % (ctx // 2) for i in range(n)]
    pages = [-(-(x + T) // 16) for x in lens]
    table = torch.full((n, max(pages)), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).int(), 0
    for i, k in enumerate(pages):
        table[i, :k], at = order[at:at + k], at + k
    k = torch.randn(sum(pages), 16, kv, d, device="cuda")
    cache = cv.PagedCache(k, torch.ones_like(k), table.cuda())
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.zeros(n, T, H, d, device="cuda")
    for _ in range(5):
        out = torch.zeros_like(q)
        cv.tree_attention(q, out, cache, lens)
        assert float((out - 1).abs().max()) <= 2.0 ** -20
