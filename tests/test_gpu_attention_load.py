"""Tree attention with every SM reading: many sequences whose last tiles begin while the tiles before them are still on their way."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPES = [  # sequences, longest context, heads, kv heads, head size, drafts
    (160, 1500, 32, 4, 128, 8), (64, 1500, 64, 8, 128, 17), (160, 1500, 16, 8, 64, 4), (64, 1500, 32, 8, 64, 40),
    (96, 1200, 8, 4, 192, 4), (96, 1200, 8, 4, 256, 4), (160, 300, 8, 1, 128, 4),
]


def _state(shape, g):
    n, ctx, H, kv, d, T = shape
    page = 16
    lens = [ctx - i * 41 % (ctx // 2) for i in range(n)]
    pages = [-(-(x + T) // page) for x in lens]
    table = torch.full((n, max(pages)), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).int(), 0
    for i, k in enumerate(pages):
        table[i, :k], at = order[at:at + k], at + k
    k = torch.randn(sum(pages), page, kv, d, generator=g, device="cuda", dtype=BF)
    return k, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_every_key_counts_once(cuda_lib, shape):
    """Queries of zero weigh all keys alike, and values of one then give exactly one: numerator and denominator are the same
    number of keys, whole numbers below 2^24, whatever the tiles and parts.  A page of V left out is 16 of at most
    1540 keys, 2.6 roundings of bf16 near one (2^-8)."""
    cv = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(3)
    k, table, lens = _state(shape, g)
    n, _, H, _, d, T = shape
    cache = cv.PagedCache(k, torch.ones_like(k), table)
    q = torch.zeros(n, T, H, d, dtype=BF, device="cuda")
    for _ in range(12):
        out = torch.zeros_like(q)
        cv.tree_attention(q, out, cache, lens)
        assert torch.equal(out, torch.ones_like(out))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_repeats(cuda_lib, shape):
    """The split of the work and the order of the sums depend on the lengths alone."""
    cv = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(4)
    k, table, lens = _state(shape, g)
    n, _, H, _, d, T = shape
    cache = cv.PagedCache(k, torch.randn(k.shape, generator=g, device="cuda", dtype=BF), table)
    q = torch.randn(n, T, H, d, generator=g, device="cuda", dtype=BF)
    err = torch.zeros(n, dtype=torch.int32, device="cuda")
    first = torch.zeros_like(q)
    cv.tree_attention(q, first, cache, lens, err=err)
    for _ in range(12):
        out = torch.zeros_like(q)
        cv.tree_attention(q, out, cache, lens, err=err)
        assert torch.equal(out, first) and not bool(err.any())
