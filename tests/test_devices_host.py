"""Tensors on other devices than the current one are refused before anything is launched (no GPU: CPU tensors that
say they are on a device, and a library that fails the test when it is called)."""
from __future__ import annotations

import pytest
import torch

import spec_decode_verify_gb300 as cv


class OnDevice(torch.Tensor):
    index = 0

    def get_device(self):
        return self.index

    @property
    def is_cuda(self):
        return self.index >= 0


def put(t, index):
    t = t.as_subclass(OnDevice)
    t.index = index
    return t


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    def fail(*_):
        raise AssertionError("the library was called")

    monkeypatch.setattr(cv, "load_library", fail)
    monkeypatch.setattr(cv, "_current_device", lambda: 0)


def layer_calls():
    bf = torch.bfloat16
    q, v, g = torch.zeros(2, 3, 1, 16, dtype=bf), torch.zeros(2, 3, 2, 8, dtype=bf), torch.zeros(2, 3, 2)
    i32 = torch.zeros(2, dtype=torch.int32)
    step = dict(q=q, k=q.clone(), v=v, log_decay=g, state=torch.zeros(2, 2, 16, 8), out=v.clone(), gain=g.clone(),
                skip=torch.zeros(2), cache_idx=i32, has_initial_state=i32.clone(), err=i32.clone())
    flat = {n: t.flatten(0, 1) if n in ("q", "k", "v", "log_decay", "out", "gain") else t for n, t in step.items()}
    drafts = dict(k=q.clone(), v=v.clone(), log_decay=g.clone(), accept_len=i32.clone(), gain=g.clone())
    y = torch.zeros(2, 8)
    norm = dict(y=y, out=y.clone(), gate=y.clone(), post_weight=torch.zeros(8), residual=y.clone(), residual_out=y.clone(),
                channel_scale=torch.zeros(8), pre_weight=torch.zeros(8))
    cu = torch.tensor([0, 3, 6], dtype=torch.int32)
    return {
        "step": (step, lambda t: cv.linattn_step(**t)),
        "prefill": ({**flat, "cu_seqlens": cu, "workspace": torch.zeros(256, dtype=torch.uint8)},
                    lambda t: cv.linattn_prefill(**t, max_seqlen=3)),
        "commit": ({**drafts, "state": torch.zeros(2, 2, 16, 8)},
                   lambda t: cv.linattn_commit(cv.LinattnDrafts(**{n: x for n, x in t.items() if n != "state"}), t["state"])),
        "norm": (norm, lambda t: cv.block_norm(**t, group=8)),
    }


def conv_calls():
    i32 = torch.zeros(2, dtype=torch.int32)
    x, state, weight = torch.zeros(2, 3, 16), torch.zeros(2, 16, 3), torch.zeros(16, 4)
    verify = dict(x=x, conv_state=state, weight=weight, bias=torch.zeros(16), out=x.clone(), window=torch.zeros(2, 16, 5),
                  cache_idx=i32, state_off=i32.clone(), err=i32.clone())
    commit = dict(conv_state=state, window=torch.zeros(2, 16, 5), accept_len=i32.clone(), cache_idx=i32, err=i32.clone())
    flat = torch.zeros(6, 16)
    prefill = dict(x=flat, conv_state=state, weight=weight, bias=torch.zeros(16), out=flat.clone(),
                   cu_seqlens=torch.tensor([0, 3, 6], dtype=torch.int32), cache_idx=i32, has_initial_state=i32.clone(),
                   err=i32.clone())
    return {
        "conv_verify": (verify, lambda t: cv.conv_verify(**t, layout="dedup", qk_channels=8, head_dim=8)),
        "conv_commit": (commit, lambda t: cv.conv_commit(**t, layout="dedup", T=3, width=4)),
        "conv_prefill": (prefill, lambda t: cv.conv_prefill(**t, max_seqlen=3, qk_channels=8, head_dim=8)),
    }


CALLS = {**layer_calls(), **conv_calls()}


def refused(call, on, match):
    tensors, run = call
    with pytest.raises(ValueError, match=match):
        run({n: put(t, on(n)) for n, t in tensors.items()})


@pytest.mark.parametrize("name", CALLS)
def test_everything_on_the_current_device_reaches_the_library(name, monkeypatch):
    monkeypatch.setattr(cv, "_stream_of", lambda *_: 0)
    monkeypatch.setattr(cv, "_stream_ptr", lambda *_: 0)
    tensors, run = CALLS[name]
    with pytest.raises(AssertionError, match="library was called"):
        run({n: put(t, 0) for n, t in tensors.items()})


@pytest.mark.parametrize("name", CALLS)
def test_another_device_than_the_current_one(name):
    refused(CALLS[name], lambda n: 1, "current device is cuda:0")


@pytest.mark.parametrize("name,tensor", [(name, t) for name in CALLS for t in CALLS[name][0]])
def test_one_tensor_elsewhere(name, tensor):
    refused(CALLS[name], lambda n: 1 if n == tensor else 0, "one device|current device")
    refused(CALLS[name], lambda n: -1 if n == tensor else 0, "CUDA tensor")
