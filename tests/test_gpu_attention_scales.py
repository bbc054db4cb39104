"""Scales of any sign and size, and sequences that read one slot at once."""
from __future__ import annotations

import pytest
import torch

import attn_reference as ref
from test_gpu_attention import BF, F32, call, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-42, 1e-30, 3.0, -0.0])
def test_scales(cuda_lib, scale, dtype):
    x = make([0, 70, 300], [5] * 3, 5, 2, 3, 64, 16, dtype, tree=True)
    out, err = call(cuda_lib, x, scale=scale)
    assert err == [0] * 3
    for s, L in enumerate(x["lens"]):
        row = x["table"][int(x["slots"][s])]
        K, V = ref.gather(x["k"], row, L + 5), ref.gather(x["v"], row, L + 5)
        want, size, top = ref.attention(x["q"][s].double(), K, V, L, x["parents"][s], scale)
        bound = ref.attention_bound(dtype, want, size, top.abs(), L + 5, 64)
        assert bool(((out[s].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_slot_read_by_many(cuda_lib, dtype):
    """Sequences of one slot, each of a length of its own."""
    x = make([400], [3], 3, 2, 4, 128, 16, dtype)
    n = 9
    x["slots"] = x["slots"].repeat(n)
    x["lens"], x["counts"], x["parents"] = [400 - 37 * i for i in range(n)], [3] * n, x["parents"] * n
    x["q"] = torch.randn(n, 3, 8, 128, generator=torch.Generator().manual_seed(1)).to(dtype)
    out, err = call(cuda_lib, x)
    assert err == [0] * n
    row = x["table"][int(x["slots"][0])]
    for s, L in enumerate(x["lens"]):
        K, V = ref.gather(x["k"], row, L + 3), ref.gather(x["v"], row, L + 3)
        want, size, top = ref.attention(x["q"][s].double(), K, V, L, x["parents"][s], 128 ** -0.5)
        assert bool(((out[s].double() - want).abs() <= ref.attention_bound(dtype, want, size, top, L + 3, 128)).all())
