"""Arguments of the operators beside the conv, without a GPU: the binding's structs, and what it refuses."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import spec_decode_verify_gb300 as cv
from spec_decode_verify_gb300 import build as cvbuild
from test_layer_host import tensors

HEADER = os.path.join(cvbuild.INCLUDE, "convverify.h")


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    mirrors = {"cv_linattn_tokens": cv.LinattnTokens, "cv_linattn_args": cv.LinattnArgs, "cv_norm_args": cv.NormArgs}
    lines = ["#include <stddef.h>", "#include <stdio.h>", f'#include "{HEADER}"', "int main(void) {"]
    for name, py in mirrors.items():
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in py._fields_]
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
    (tmp_path / "layout.c").write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run([cc, "-std=c99", "-o", str(tmp_path / "layout"), str(tmp_path / "layout.c")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    want = "".join("".join(f"{name} {f} {getattr(py, f).offset}\n" for f, _ in py._fields_) +
                   f"{name} size {ctypes.sizeof(py)}\n" for name, py in mirrors.items())
    assert got == want


def test_packed_arguments_land_in_their_fields():
    t = tensors()
    a = cv.make_linattn_args(t["q"], t["k"], t["v"], t["g"], t["state"], t["out"], n_seq=2, check_device=False,
                             update_state=True, wait_polls=-5, workspace=torch.zeros(512, dtype=torch.uint8))
    assert (a.update_state, a.wait_polls, a.workspace_bytes, a.tok.T, a.prev.T) == (1, -5, 512, 3, 0)
    assert a.out == t["out"].data_ptr() and a.state == t["state"].data_ptr() and a.tok.log_decay == t["g"].data_ptr()


@pytest.fixture(scope="module")
def lib():
    cvbuild.build()
    return cv.load_library()


def prompt_args(dtype, total, dk, dv, nh, shift):
    """Arguments of one prompt whose out rows start `shift` elements past a 16-byte boundary."""
    x = torch.zeros(total, 1, dk, dtype=dtype)
    v = torch.zeros(total, nh, dv, dtype=dtype)
    out = torch.zeros(total * nh * dv + 8, dtype=dtype)[shift:shift + total * nh * dv].view(total, nh, dv)
    cu = torch.tensor([0, total], dtype=torch.int32)
    a = cv.make_linattn_args(x, x.clone(), v, torch.zeros(total, nh), torch.zeros(1, nh, dk, dv), out, n_seq=1, cu=cu, T=total,
                             check_device=False)
    a.keep = (x, v, out, cu)
    return a


def workspace(lib, a):
    n = ctypes.c_int64(-1)
    assert lib.cv_linattn_workspace(ctypes.byref(a), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("total,dk,dv,nh", [(300, 64, 64, 1), (1000, 128, 128, 2), (700, 8, 16, 1), (4000, 64, 128, 1),
                                            (20000, 128, 64, 3), (40, 64, 64, 1)])
def test_a_size_asked_for_without_pointers_is_enough_for_any(lib, dtype, total, dk, dv, nh):
    needs = [workspace(lib, prompt_args(dtype, total, dk, dv, nh, shift)) for shift in (0, 1, 2, 4)]
    for null in (("out",), ("state",), ("q", "k", "v"), ("q", "k", "v", "out", "state")):
        a = prompt_args(dtype, total, dk, dv, nh, 0)
        for name in null:
            setattr(a if name in ("out", "state") else a.tok, name, None)
        assert workspace(lib, a) >= max(needs)


def test_a_stride_over_one_channel_does_not_matter():
    """Heads of one channel: the innermost stride is never used, whatever a transpose or an expansion left there."""
    def odd(*shape):
        return torch.zeros(*shape[:-1], 7)[..., 3:4].as_strided(shape, (*torch.zeros(*shape).stride()[:-1], 5))

    for dk, dv in ((1, 1), (1, 4), (4, 1)):
        q, v = (odd if dk == 1 else torch.zeros)(2, 3, 1, dk), (odd if dv == 1 else torch.zeros)(2, 3, 2, dv)
        out = (odd if dv == 1 else torch.zeros)(2, 3, 2, dv)
        a = cv.make_linattn_args(q, q, v, torch.zeros(2, 3, 2), torch.zeros(2, 2, dk, dv), out, n_seq=2, check_device=False)
        assert (a.dk, a.dv) == (dk, dv)
    with pytest.raises(ValueError):
        wide = torch.zeros(2, 3, 1, 8)[..., ::2]
        cv.make_linattn_args(wide, wide, torch.zeros(2, 3, 2, 4), torch.zeros(2, 3, 2), torch.zeros(2, 2, 4, 4),
                             torch.zeros(2, 3, 2, 4), n_seq=2, check_device=False)
