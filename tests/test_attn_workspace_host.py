"""Workspace of the tree attention: the size for pointers not known yet is enough for a call with any alignment of them."""
from __future__ import annotations

import ctypes

import pytest

import spec_decode_verify_gb300 as cv


@pytest.mark.parametrize("dtype", [cv.F32, cv.BF16])
@pytest.mark.parametrize("T,n_heads,head_dim,page", [(1, 2, 128, 16), (1, 16, 64, 16), (4, 4, 256, 32), (17, 16, 128, 16), (2, 2, 24, 5)])
def test_unknown_pointers(dtype, T, n_heads, head_dim, page):
    lib = cv.load_library()
    a = cv.TreeAttentionArgs()
    c = a.cache
    c.n_layers, c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.n_slots, c.max_pages = 1, 4096, page, 2, head_dim, 64, 64
    c.dtype, c.table_stride = dtype, 64
    c.k_head_stride = c.v_head_stride = head_dim
    c.k_row_stride = c.v_row_stride = 2 * head_dim
    c.k_page_stride = c.v_page_stride = 2 * head_dim * page
    a.n_seq, a.T, a.n_heads, a.scale = 40, T, n_heads, 1.0
    a.q_head_stride = a.out_head_stride = head_dim
    a.q_tok_stride = a.out_tok_stride = n_heads * head_dim
    a.q_seq_stride = a.out_seq_stride = n_heads * head_dim * T

    def need(q, k, v):
        a.q, c.k, c.v = q, k, v
        n = ctypes.c_int64(-1)
        assert lib.cv_tree_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == 0
        return n.value

    at = 1 << 20
    most = need(None, None, None)
    sizes = {need(at + x, at + y, at + z) for x in (0, 4) for y in (0, 4) for z in (0, 4)}
    assert most >= max(sizes) > 0


@pytest.mark.parametrize("page,pages,status", [(1, 2 ** 31 - 1, -3), (1, 2 ** 31 - 255, -3), (1, 2 ** 31 - 256, 0), (128, 2 ** 24 - 2, 0),
                                               (128, 2 ** 24 - 1, -3), (65536, 32767, 0), (65536, 32768, -3)])
def test_longest_tables(page, pages, status):
    """A tile that begins within a table's tokens ends below 2^31."""
    a, n = cv.TreeAttentionArgs(), ctypes.c_int64()
    c = a.cache
    c.n_layers, c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.n_slots, c.max_pages = 1, 4, page, 1, 8, 1, pages
    a.n_seq, a.T, a.n_heads, a.scale = 1, 1, 1, 1.0
    assert cv.load_library().cv_tree_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == status
