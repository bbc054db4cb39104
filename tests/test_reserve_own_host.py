"""Growth with the slots' lengths, on the host: refusals of the library and the binding."""
from __future__ import annotations

import ctypes

import pytest
import torch

import spec_decode_verify_gb300 as cv
from test_attn_host import cache_of, tensors
from test_devices_host import put


def args(t, **kw):
    return cv.make_cache_pages_args(cache_of(t), 2, idx=t["idx"], n_tokens=t["tok"], err=t["err"], cache_len=t["len"], **kw)


@pytest.mark.parametrize("over,status", [(dict(err="cache_len"), -10), (dict(v="k"), -10), (dict(n_layers=4096, n_kv_heads=4096, head_dim=255), -3)])
def test_refusals(over, status):
    t = tensors()
    a = args(t, check_device=False)
    assert a.cache_len == t["len"].data_ptr()
    for name, x in over.items():
        if name == "v":
            a.cache.v = a.cache.k
        else:
            setattr(a if name == "err" else a.cache, name, getattr(a, x) if isinstance(x, str) else x)
    assert cv.load_library().cv_cache_reserve(ctypes.byref(a), None) == status


def test_binding(monkeypatch):
    with pytest.raises(ValueError):
        args({**tensors(), "len": torch.zeros(2)}, check_device=False)
    with pytest.raises(ValueError):
        args({**tensors(), "len": torch.zeros(1, dtype=torch.int32)}, check_device=False)
    monkeypatch.setattr(cv, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="device"):
        args({n: put(x, int(n == "len")) for n, x in tensors().items()}, check_device=True)
