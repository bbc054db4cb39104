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
