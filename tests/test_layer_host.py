"""Host-side refusals of the operators beside the conv (no GPU): the library rejects invalid arguments with
the documented status before anything is launched, and the binding rejects shapes and types."""
from __future__ import annotations

import ctypes

import pytest
import torch

import spec_decode_verify_gb300 as cv
from spec_decode_verify_gb300 import build as cvbuild


@pytest.fixture(scope="module")
def lib():
    cvbuild.build()
    return cv.load_library()


def tensors(n=2, T=3, nq=1, nh=2, dk=16, dv=8, dtype=torch.bfloat16):
    return dict(q=torch.zeros(n, T, nq, dk, dtype=dtype), k=torch.zeros(n, T, nq, dk, dtype=dtype),
                v=torch.zeros(n, T, nh, dv, dtype=dtype), g=torch.zeros(n, T, nh), state=torch.zeros(n, nh, dk, dv),
                out=torch.zeros(n, T, nh, dv, dtype=dtype), accept=torch.zeros(n, dtype=torch.int32))


def step_args(t, prev=False, **over):
    d = cv.LinattnDrafts(t["k"], t["v"], t["g"], t["accept"]) if prev else None
    a = cv.make_linattn_args(t["q"], t["k"], t["v"], t["g"], t["state"], t["out"], n_seq=t["q"].shape[0], prev=d,
                             check_device=False)
    a.keep = t
    for k, v in over.items():
        part, _, field = k.partition("__")
        setattr(getattr(a, part), field, v) if field else setattr(a, k, v)
    return a


STEP_ERRORS = [
    (dict(dtype=7), -6), (dict(n_seq=-1), -3), (dict(n_seq=65536), -3), (dict(n_slots=0), -3), (dict(n_heads=0), -3),
    (dict(n_heads=4097, n_qk_heads=1), -3), (dict(dk=0), -7), (dict(dk=257), -7), (dict(dv=0), -7), (dict(dv=257), -7),
    (dict(n_qk_heads=0), -7), (dict(n_heads=3, n_qk_heads=2), -7), (dict(tok__T=-1), -4), (dict(tok__T=129), -4),
    (dict(prev__T=129), -4), (dict(prev__T=-1), -4), (dict(tok__q_tok_stride=-1), -9), (dict(tok__gain_seq_stride=-2), -9),
    (dict(prev__v_head_stride=-1), -9), (dict(out_tok_stride=-1), -9), (dict(state_head_stride=127), -9),
    (dict(state_slot_stride=5), -9), (dict(state=None), -2), (dict(tok__q=None), -2), (dict(tok__log_decay=None), -2),
    (dict(out=None), -2), (dict(accept_len=None), -2), (dict(prev__k=None), -2)]


@pytest.mark.parametrize("over,status", STEP_ERRORS)
def test_step_refusals(lib, over, status):
    a = step_args(tensors(), prev=True, **over)
    assert lib.cv_linattn_step(ctypes.byref(a), None) == status
    assert cv.status_string(status) not in ("", "unknown status")


def test_step_alias_and_null(lib):
    t = tensors()
    for name in ("q", "k", "v", "log_decay"):
        a = step_args(t)
        a.out = getattr(a.tok, name)
        assert lib.cv_linattn_step(ctypes.byref(a), None) == -10
    assert lib.cv_linattn_step(None, None) == -1
    a = step_args(t, tok__cu=a.out, tok__total_tokens=-1)
    assert lib.cv_linattn_step(ctypes.byref(a), None) == -3


def test_nothing_to_do_is_ok_without_a_gpu(lib):
    a = step_args(tensors(), n_seq=0)
    assert lib.cv_linattn_step(ctypes.byref(a), None) == 0
    assert lib.cv_linattn_prefill(ctypes.byref(a), None) == 0
    y = torch.zeros(0, 8)
    assert lib.cv_block_norm(ctypes.byref(cv.make_norm_args(y, y.clone(), group=8, check_device=False)), None) == 0


def test_prefill_refusals(lib):
    a = step_args(tensors())
    assert lib.cv_linattn_prefill(ctypes.byref(a), None) == -2  # cu is required
    a = step_args(tensors(), tok__T=-3)
    assert lib.cv_linattn_prefill(ctypes.byref(a), None) == -4
    n = ctypes.c_int64(-1)
    assert lib.cv_linattn_workspace(None, ctypes.byref(n)) == -1
    assert lib.cv_linattn_workspace(ctypes.byref(step_args(tensors())), None) == -2
    assert lib.cv_linattn_workspace(ctypes.byref(step_args(tensors())), ctypes.byref(n)) == 0 and n.value >= 0


def norm_args(**over):
    t = dict(y=torch.zeros(4, 32), out=torch.zeros(4, 32), gate=torch.zeros(4, 32), residual=torch.zeros(4, 32),
             residual_out=torch.zeros(4, 32), post_weight=torch.zeros(8), pre_weight=torch.zeros(32),
             channel_scale=torch.zeros(32))
    a = cv.make_norm_args(t["y"], t["out"], group=8, check_device=False, **{k: v for k, v in t.items() if k not in ("y", "out")})
    a.keep = t
    for k, v in over.items():
        setattr(a, k, v(a) if callable(v) else v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(dtype=5), -6), (dict(residual_dtype=1), -6), (dict(rows=-1), -3), (dict(dim=0), -3), (dict(dim=65537), -3),
    (dict(group=-1), -7), (dict(group=5), -7), (dict(group=0), -7), (dict(gate_act=2), -8), (dict(y_stride=-1), -9),
    (dict(out_stride=31), -9), (dict(residual_out_stride=0), -9), (dict(y=None), -2), (dict(residual_out=None), -2),
    (dict(residual=None, out=None), -2), (dict(out=lambda a: a.residual), -10), (dict(out=lambda a: a.residual_out), -10),
    (dict(out=lambda a: a.y, out_stride=40), -10), (dict(residual_out=lambda a: a.gate), -10),
    (dict(residual_out=lambda a: a.residual, residual_out_stride=33), -10)])
def test_norm_refusals(lib, over, status):
    assert lib.cv_block_norm(ctypes.byref(norm_args(**over)), None) == status


def test_norm_group_count_that_does_not_fit(lib):
    y = torch.zeros(1, 65536)
    a = cv.make_norm_args(y, y.clone(), group=1, residual=y.clone(), residual_out=y.clone(), check_device=False)
    assert lib.cv_block_norm(ctypes.byref(a), None) == -12
    assert lib.cv_block_norm(None, None) == -1


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(2, 3, 16)), dict(k=torch.zeros(2, 3, 1, 15, dtype=torch.bfloat16)),
    dict(v=torch.zeros(2, 4, 2, 8, dtype=torch.bfloat16)), dict(g=torch.zeros(2, 3, 1)), dict(state=torch.zeros(2, 2, 16, 9)),
    dict(state=torch.zeros(2, 2, 8, 16).transpose(2, 3)), dict(out=torch.zeros(2, 3, 2, 4, dtype=torch.bfloat16)),
    dict(out=torch.zeros(2, 3, 2, 8)), dict(state=torch.zeros(2, 2, 16, 8).half())])
def test_binding_shapes(change):
    t = {**tensors(), **change}
    with pytest.raises((ValueError, TypeError)):
        cv.make_linattn_args(t["q"], t["k"], t["v"], t["g"], t["state"], t["out"], n_seq=2, check_device=False)


@pytest.mark.parametrize("change", [dict(g=torch.zeros(2, 3, 2).double()), dict(v=torch.zeros(2, 3, 2, 8)),
                                    dict(q=torch.zeros(2, 3, 1, 16).half(), k=torch.zeros(2, 3, 1, 16).half(),
                                         v=torch.zeros(2, 3, 2, 8).half(), out=torch.zeros(2, 3, 2, 8).half())])
def test_binding_types(change):
    t = {**tensors(), **change}
    with pytest.raises(TypeError):
        cv.make_linattn_args(t["q"], t["k"], t["v"], t["g"], t["state"], t["out"], n_seq=2, check_device=False)


def test_binding_index_arrays_and_packed_rows():
    t = tensors()

    def build(n_seq=2, **kw):
        return cv.make_linattn_args(t["q"], t["k"], t["v"], t["g"], t["state"], t["out"], n_seq=n_seq, check_device=False,
                                    **kw)

    build(cache_idx=torch.zeros(2, dtype=torch.int32))
    for kw in (dict(cache_idx=torch.zeros(2)), dict(err=torch.zeros(1, dtype=torch.int32)), dict(n_seq=3), dict(T=4),
               dict(skip=torch.zeros(3)), dict(skip=torch.zeros(2).double()),
               dict(prev=cv.LinattnDrafts(t["k"][:1], t["v"][:1], t["g"][:1], t["accept"])),
               dict(prev=cv.LinattnDrafts(t["k"], t["v"], t["g"], t["accept"].long()))):
        with pytest.raises((ValueError, TypeError)):
            build(**kw)
    p = {k: v.flatten(0, 1) if v.dim() > 2 and k != "state" else v for k, v in t.items()}
    cu = torch.tensor([0, 2, 6], dtype=torch.int32)
    ok = dict(n_seq=2, check_device=False)
    cv.make_linattn_args(p["q"], p["k"], p["v"], p["g"], t["state"], p["out"], cu=cu, T=4, **ok)
    for bad in (dict(cu=cu), dict(cu=cu.long(), T=4), dict(cu=cu[:2], T=4)):
        with pytest.raises(ValueError):
            cv.make_linattn_args(p["q"], p["k"], p["v"], p["g"], t["state"], p["out"], **bad, **ok)


def test_there_is_no_cpu_path():
    t = tensors()
    with pytest.raises(ValueError, match="CUDA tensor"):
        cv.linattn_step(t["q"], t["k"], t["v"], t["g"], t["state"], t["out"])
    with pytest.raises(ValueError, match="CUDA tensor"):
        cv.block_norm(torch.zeros(2, 8), torch.zeros(2, 8), group=8)


@pytest.mark.parametrize("kw", [
    dict(gate=torch.zeros(4, 31)), dict(gate_act="tanh", gate=torch.zeros(4, 32)), dict(post_weight=torch.zeros(7), group=8),
    dict(pre_weight=torch.zeros(32)), dict(residual=torch.zeros(4, 32)), dict(residual_out=torch.zeros(4, 32)),
    dict(post_weight=torch.zeros(8).bfloat16(), group=8), dict(residual=torch.zeros(4, 32), residual_out=torch.zeros(4, 32).bfloat16()),
    dict(gate=torch.zeros(32, 4).t())])
def test_norm_binding(kw):
    with pytest.raises((ValueError, TypeError)):
        cv.make_norm_args(torch.zeros(4, 32), torch.zeros(4, 32), check_device=False, **kw)
