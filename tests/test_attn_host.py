"""Attention layers' operators without a GPU: struct layouts, refusals of the library and of the binding, devices."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import spec_decode_verify_gb300 as cv
from spec_decode_verify_gb300 import build as cvbuild
from test_devices_host import put

HEADER = os.path.join(cvbuild.INCLUDE, "convverify.h")
MIRRORS = {"cv_cache": cv.Cache, "cv_tree_attention_args": cv.TreeAttentionArgs, "cv_draft_verify_args": cv.DraftVerifyArgs,
           "cv_qk_norm_rope_args": cv.QkNormRopeArgs, "cv_cache_compact_args": cv.CacheCompactArgs,
           "cv_cache_pages_args": cv.CachePagesArgs}


@pytest.fixture(scope="module")
def lib():
    cvbuild.build()
    return cv.load_library()


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stddef.h>", "#include <stdio.h>", f'#include "{HEADER}"', "int main(void) {"]
    for name, py in MIRRORS.items():
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in py._fields_]
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
    (tmp_path / "layout.c").write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run([cc, "-std=c99", "-o", str(tmp_path / "layout"), str(tmp_path / "layout.c")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    want = "".join("".join(f"{name} {f} {getattr(py, f).offset}\n" for f, _ in py._fields_) +
                   f"{name} size {ctypes.sizeof(py)}\n" for name, py in MIRRORS.items())
    assert got == want


def tensors(n=2, T=3, H=4, kv=2, d=16, page=8, pages=5, dtype=torch.bfloat16):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=torch.zeros(n, T, H, d, dtype=dtype), out=torch.zeros(n, T, H, d, dtype=dtype),
                k=torch.zeros(n, T, kv, d, dtype=dtype), v=torch.zeros(n, T, kv, d, dtype=dtype),
                kc=torch.zeros(pages, page, kv, d, dtype=dtype), vc=torch.zeros(pages, page, kv, d, dtype=dtype),
                table=i32(n, 4), held=i32(n), refs=i32(pages), len=i32(n), parent=i32(n, T), idx=i32(n), err=i32(n),
                probs=torch.zeros(n, T, 10), tokens=i32(n, T), u=torch.zeros(n, T + 1), accept=i32(n), new=i32(n, T), path=i32(n, T),
                node=i32(n), dprobs=torch.zeros(n, T, 10), cs=torch.zeros(9, d), w=torch.zeros(d, dtype=dtype), src=i32(n), tok=i32(n),
                new_len=i32(n))


def cache_of(t):
    return cv.PagedCache(t["kc"], t["vc"], t["table"], held=t["held"], refs=t["refs"])


def struct_of(name, t, check_device=False):
    c = cache_of(t)
    kw = dict(check_device=check_device)
    a = {"attention": lambda: cv.make_tree_attention_args(t["q"], t["out"], c, t["len"], parent=t["parent"], cache_idx=t["idx"], err=t["err"], **kw),
         "verify": lambda: cv.make_draft_verify_args(t["probs"], t["tokens"], t["u"], t["accept"], t["new"], draft_probs=t["dprobs"],
                                                     path=t["path"], accept_node=t["node"], err=t["err"], **kw),
         "rope": lambda: cv.make_qk_norm_rope_args(t["q"], t["k"], t["out"], v=t["v"], cos_sin=t["cs"], q_weight=t["w"], k_weight=t["w"],
                                                   cache=c, cache_len=t["len"], err=t["err"], **kw),
         "compact": lambda: cv.make_cache_compact_args(c, t["len"], t["path"], t["accept"], new_len=t["new_len"], err=t["err"], **kw),
         "reserve": lambda: cv.make_cache_pages_args(c, 2, idx=t["idx"], n_tokens=t["tok"], err=t["err"], **kw),
         "fork": lambda: cv.make_cache_pages_args(c, 2, idx=t["idx"], src_idx=t["src"], n_tokens=t["tok"], err=t["err"], **kw),
         "free": lambda: cv.make_cache_pages_args(c, 2, idx=t["idx"], err=t["err"], **kw)}[name]()
    a.keep = t
    return a


ENTRY = {"attention": "cv_tree_attention", "verify": "cv_draft_verify", "rope": "cv_qk_norm_rope", "compact": "cv_cache_compact",
         "reserve": "cv_cache_reserve", "fork": "cv_cache_fork", "free": "cv_cache_free"}
CACHE = [(dict(cache__dtype=3), -6), (dict(cache__n_layers=0), -3), (dict(cache__n_layers=4097), -3), (dict(cache__n_pages=0), -3),
         (dict(cache__page_size=0), -3), (dict(cache__page_size=65537), -3), (dict(cache__n_slots=0), -3), (dict(cache__max_pages=0), -3),
         (dict(cache__max_pages=1 << 28), -3), (dict(cache__k_row_stride=-1), -9), (dict(cache__v_head_stride=-1), -9),
         (dict(cache__table_stride=3), -9), (dict(cache__k=None), -2), (dict(n_seq=-1), -3)]
REFUSED = {
    "attention": CACHE + [(dict(n_seq=65536), -3), (dict(n_heads=0), -3), (dict(n_heads=4098), -3), (dict(n_heads=5), -7), (dict(T=0), -4),
                          (dict(T=129), -4), (dict(cache__head_dim=0), -7), (dict(cache__head_dim=257), -7), (dict(q_tok_stride=-1), -9),
                          (dict(out_head_stride=-1), -9), (dict(q=None), -2), (dict(out=None), -2), (dict(cache_len=None), -2),
                          (dict(cache__page_table=None), -2), (dict(out="q"), -10), (dict(cu_draft="q", total_tokens=-1), -3)],
    "verify": [(dict(dtype=2), -6), (dict(n_seq=-1), -3), (dict(n_seq=65536), -3), (dict(vocab=0), -3), (dict(vocab=(1 << 24) + 1), -3),
               (dict(T=0), -4), (dict(T=129), -4), (dict(parent="tokens"), -8), (dict(probs_tok_stride=-1), -9),
               (dict(draft_seq_stride=-1), -9), (dict(probs=None), -2), (dict(tokens=None), -2), (dict(uniforms=None), -2),
               (dict(accept_len=None), -2), (dict(out_tokens=None), -2), (dict(out_tokens="tokens"), -10), (dict(path="out_tokens"), -10),
               (dict(accept_node="accept_len"), -10), (dict(cu_draft="probs", total_tokens=-2), -3)],
    "rope": CACHE[1:] + [(dict(dtype=2), -6), (dict(dtype=0), -6), (dict(n_seq=65536), -3), (dict(n_heads=-1), -3), (dict(n_heads=4097), -3),
                         (dict(n_kv_heads=4097), -3), (dict(n_kv_heads=1), -7), (dict(T=-1), -4), (dict(head_dim=0), -7),
                         (dict(head_dim=257), -7), (dict(rot_dim=3), -7), (dict(rot_dim=18), -7), (dict(q_seq_stride=-1), -9),
                         (dict(cos_sin_stride=8), -9), (dict(n_positions=0), -9), (dict(q=None), -2), (dict(q_out=None), -2), (dict(k=None), -2),
                         (dict(cos_sin=None), -2), (dict(cache_len=None), -2), (dict(q_out="k"), -10), (dict(q_out="q", q_out_tok_stride=65), -10),
                         (dict(k_out="q_out"), -10)],
    "compact": CACHE + [(dict(n_seq=65536), -3), (dict(T=0), -4), (dict(T=129), -4), (dict(cache_len=None), -2), (dict(path=None), -2),
                        (dict(accept_len=None), -2), (dict(new_len="cache_len"), -10), (dict(err="accept_len"), -10), (dict(err="new_len"), -10)],
    "reserve": CACHE + [(dict(n_seq=4097), -3), (dict(n_tokens=None), -2), (dict(cache__held=None), -2), (dict(cache__refs=None), -2),
                        (dict(err="n_tokens"), -10), (dict(err="idx"), -10)],
    "fork": CACHE + [(dict(src_idx=None), -2), (dict(n_tokens=None), -2), (dict(err="src_idx"), -10)],
    "free": CACHE + [(dict(n_seq=4097), -3), (dict(cache__held=None), -2), (dict(err="idx"), -10)],
}


@pytest.mark.parametrize("name,over,status", [(n, o, s) for n, cases in REFUSED.items() for o, s in cases])
def test_refusals(lib, name, over, status):
    a = struct_of(name, tensors())
    for k, v in over.items():
        part, _, field = k.partition("__")
        to = getattr(a, part) if field else a
        setattr(to, field or k, getattr(a, v) if isinstance(v, str) else v)
    assert getattr(lib, ENTRY[name])(ctypes.byref(a), None) == status
    assert cv.status_string(status) not in ("", "unknown status")


@pytest.mark.parametrize("name", ENTRY)
def test_nothing_to_do_and_no_arguments(lib, name):
    a = struct_of(name, tensors())
    a.n_seq = 0
    assert getattr(lib, ENTRY[name])(ctypes.byref(a), None) == 0
    assert getattr(lib, ENTRY[name])(None, None) == -1


def test_workspace_sizes(lib):
    t = tensors()
    a = struct_of("attention", t)
    n = ctypes.c_int64(-1)
    assert lib.cv_tree_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0  # one tile holds all keys
    assert lib.cv_tree_attention_workspace(ctypes.byref(a), None) == -2
    assert lib.cv_tree_attention_workspace(None, ctypes.byref(n)) == -1
    a.cache.max_pages = a.cache.table_stride = 1000
    assert lib.cv_tree_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.cv_tree_attention(ctypes.byref(a), None) == -13
    known = n.value
    a.q = a.out = a.cache.k = a.cache.v = None
    assert lib.cv_tree_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value >= known


BINDING = [("attention", dict(q=torch.zeros(2, 3, 16))), ("attention", dict(q=torch.zeros(2, 3, 4, 16))), ("attention", dict(out=torch.zeros(2, 3, 4, 8))),
           ("attention", dict(len=torch.zeros(1, dtype=torch.int32))), ("attention", dict(len=torch.zeros(2))), ("attention", dict(len=None)),
           ("attention", dict(parent=torch.zeros(2, 2, dtype=torch.int32))), ("attention", dict(kc=torch.zeros(5, 8, 2, 17, dtype=torch.bfloat16))),
           ("attention", dict(vc=torch.zeros(5, 8, 2, 16))), ("attention", dict(table=torch.zeros(2, 4))),
           ("attention", dict(table=torch.zeros(4, 2, dtype=torch.int32).T)), ("attention", dict(q=torch.zeros(2, 3, 4, 32, dtype=torch.bfloat16)[..., ::2])),
           ("verify", dict(probs=torch.zeros(2, 10))), ("verify", dict(probs=torch.zeros(2, 3, 10).half())), ("verify", dict(tokens=None)),
           ("verify", dict(u=torch.zeros(2, 3))), ("verify", dict(u=torch.zeros(2, 4).double())), ("verify", dict(new=torch.zeros(2, 4, dtype=torch.int32))),
           ("verify", dict(dprobs=torch.zeros(2, 3, 11))), ("verify", dict(probs=torch.zeros(2, 3, 20)[..., ::2], dprobs=None)),
           ("rope", dict(k=torch.zeros(2, 3, 1, 16, dtype=torch.bfloat16))), ("rope", dict(v=torch.zeros(2, 3, 2, 16))), ("rope", dict(w=torch.zeros(16))),
           ("rope", dict(cs=torch.zeros(9, 16).double())), ("rope", dict(out=torch.zeros(2, 3, 4, 16))), ("rope", dict(len=None)),
           ("compact", dict(path=torch.zeros(2, dtype=torch.int32))), ("compact", dict(accept=torch.zeros(1, dtype=torch.int32))),
           ("reserve", dict(refs=torch.zeros(4, dtype=torch.int32))), ("reserve", dict(held=None)), ("reserve", dict(tok=torch.zeros(2))),
           ("fork", dict(src=torch.zeros(3, dtype=torch.int32)))]


@pytest.mark.parametrize("name,change", BINDING)
def test_binding(name, change):
    with pytest.raises((ValueError, TypeError)):
        struct_of(name, {**tensors(), **change})


def test_a_cache_of_layers_goes_layer_by_layer():
    t = tensors()
    many = cv.PagedCache(torch.zeros(3, *t["kc"].shape), torch.zeros(3, *t["kc"].shape), t["table"])
    with pytest.raises(ValueError):
        cv.make_tree_attention_args(t["q"].float(), t["out"].float(), many, t["len"], check_device=False)
    one = many.layer(1)
    a = cv.make_tree_attention_args(t["q"].float(), t["out"].float(), one, t["len"], check_device=False)
    assert a.cache.k == many.k[1].data_ptr() and a.cache.n_layers == 1
    with pytest.raises(AttributeError):
        many.k = t["kc"]


USED = {"attention": ("q", "out", "kc", "vc", "table", "len", "parent", "idx", "err"),
        "verify": ("probs", "tokens", "u", "accept", "new", "dprobs", "path", "node", "err"),
        "rope": ("q", "k", "out", "v", "cs", "w", "kc", "vc", "table", "len", "err"),
        "compact": ("kc", "vc", "table", "len", "path", "accept", "new_len", "err"),
        "reserve": ("kc", "vc", "table", "held", "refs", "idx", "tok", "err"),
        "fork": ("kc", "vc", "table", "held", "refs", "idx", "src", "tok", "err"),
        "free": ("kc", "vc", "table", "held", "refs", "idx", "err")}


@pytest.mark.parametrize("name,tensor", [(n, t) for n, ts in USED.items() for t in ts])
def test_one_tensor_elsewhere(name, tensor, monkeypatch):
    monkeypatch.setattr(cv, "_current_device", lambda: 0)
    for index in (1, -1):
        t = {n: put(x, index if n == tensor else 0) for n, x in tensors().items()}
        with pytest.raises(ValueError, match="device|CUDA tensor"):
            struct_of(name, t, check_device=True)
    t = {n: put(x, 1) for n, x in tensors().items()}
    with pytest.raises(ValueError, match="current device is cuda:0"):
        struct_of(name, t, check_device=True)
    struct_of(name, {n: put(x, 0) for n, x in tensors().items()}, check_device=True)
