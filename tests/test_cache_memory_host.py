"""A cache's tensors that are given other memory after its handle was made: every call says so, and none uses the old addresses."""
from __future__ import annotations

import pytest
import torch

import spec_decode_verify_gb300 as cv
from test_attn_host import ENTRY, cache_of, struct_of, tensors


def make(name, t, cache, monkeypatch):
    monkeypatch.setattr("test_attn_host.cache_of", lambda _: cache)
    return struct_of(name, t)



CHANGES = {"set": lambda x: x.set_(torch.zeros_like(x)), "data": lambda x: setattr(x, "data", torch.zeros_like(x)),
           "empty": lambda x: x.untyped_storage().resize_(0), "resize": lambda x: x.resize_(64 * x.numel())}


@pytest.mark.parametrize("how", CHANGES)
@pytest.mark.parametrize("tensor", ["kc", "vc", "table", "held", "refs"])
@pytest.mark.parametrize("name", [n for n in ENTRY if n != "verify"])
def test_other_memory(name, tensor, how, monkeypatch):
    t = tensors()
    cache = cache_of(t)
    make(name, t, cache, monkeypatch)
    keep = t[tensor].clone(), t[tensor].untyped_storage()  # noqa: F841  (the old memory is not given to the new tensor)
    CHANGES[how](t[tensor])
    with pytest.raises(ValueError, match="other memory"):
        make(name, t, cache, monkeypatch)


def test_other_contents_and_a_handle_made_again(monkeypatch):
    t = tensors()
    cache = cache_of(t)
    t["kc"].fill_(1)
    t["table"].add_(1)
    assert make("attention", t, cache, monkeypatch).cache.k == t["kc"].data_ptr()
    t["kc"].data = torch.zeros_like(t["kc"])
    assert make("attention", t, cache_of(t), monkeypatch).cache.k == t["kc"].data_ptr()


def test_layers(monkeypatch):
    t = tensors()
    k = torch.zeros(3, *t["kc"].shape, dtype=t["kc"].dtype)
    cache = cv.PagedCache(k, torch.zeros_like(k), t["table"], held=t["held"], refs=t["refs"])
    one = cache.layer(2)
    k.data = torch.zeros_like(k)
    with pytest.raises(ValueError, match="other memory"):
        make("compact", t, cache, monkeypatch)
    make("attention", t, one, monkeypatch)  # a view of its own, which keeps the old memory alive
