"""Contexts that fill the longest table there is, 2^31 - 256 tokens, all of them in one page."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
TOKENS = 2 ** 31 - 256


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spare", [0, 1, 64, 700])
def test_every_key_counts_once(cuda_lib, spare, dtype):
    """Queries of zero and values of one: a block's numerator and denominator are the same whole number below 2^24 (at most 2^31 / 152), and
    the join adds both up in the same steps.  Their quotient, by a reciprocal and a product of one rounding each, is one within 2^-23, and exactly
    one in bf16."""
    cv, page = cuda_lib, 256
    k = torch.randn(1, page, 1, 64, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(dtype)
    cache = cv.PagedCache(k, torch.ones_like(k), torch.zeros(1, TOKENS // page, dtype=torch.int32, device="cuda"))
    q = torch.zeros(1, 2, 1, 64, dtype=dtype, device="cuda")
    out, err = torch.zeros_like(q), torch.full((1,), -7, dtype=torch.int32, device="cuda")
    cv.tree_attention(q, out, cache, torch.tensor([TOKENS - 2 - spare], dtype=torch.int32, device="cuda"), err=err)
    assert err.tolist() == [0] and bool(((out.float() - 1).abs() <= (2.0 ** -23 if dtype == torch.float32 else 0)).all())
    if spare == 0:
        cv.tree_attention(q, out, cache, torch.tensor([TOKENS - 1], dtype=torch.int32, device="cuda"), err=err)
        assert err.tolist() == [64]
