"""Calls without a row, on the host: nothing is launched without flags to raise, and what the flags are made of is needed."""
from __future__ import annotations

import ctypes

import spec_decode_verify_gb300 as cv
from test_attn_host import struct_of, tensors


def test_no_packed_rows():
    lib = cv.load_library()
    a = struct_of("attention", tensors())
    a.cu_draft, a.total_tokens, a.q, a.out, a.parent = a.cache_len, 0, None, None, None
    err, a.err = a.err, None
    assert lib.cv_tree_attention(ctypes.byref(a), None) == 0
    a.cache_len = None
    assert lib.cv_tree_attention(ctypes.byref(a), None) == 0
    a.err = err
    assert lib.cv_tree_attention(ctypes.byref(a), None) == -2
    r = struct_of("rope", tensors())
    r.cu, r.total_tokens, r.q, r.k, r.v, r.q_out, r.err = r.cache_len, 0, None, None, None, None, None
    assert lib.cv_qk_norm_rope(ctypes.byref(r), None) == 0
    r.cu, r.T = None, 0
    assert lib.cv_qk_norm_rope(ctypes.byref(r), None) == 0
