"""GPU tests of the block norms against their fp64 form."""
from __future__ import annotations

import pytest
import torch

from layer_reference import EPS16, EPS32, assert_within, norm

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(rows, dim, dtype, seed=0, group=0, gate=False, res=None, cs=False, pre=False, post=True, wide=0):
    rng = torch.Generator().manual_seed(seed)

    def buf(dt):
        return torch.randn(rows, dim + wide, generator=rng).to(dt)[:, :dim]

    t = dict(y=buf(DT[dtype]), gate=buf(DT[dtype]) if gate else None, residual=buf(DT[res]) if res else None)
    t["post_weight"] = (1 + 0.2 * torch.randn(group, generator=rng)).to(DT[dtype]) if group and post else None
    t["channel_scale"] = torch.rand(dim, generator=rng).to(DT[dtype]) if cs else None
    t["pre_weight"] = (1 + 0.2 * torch.randn(dim, generator=rng)).to(DT[dtype]) if pre else None
    return t


def run(cv, t, dtype, *, out=True, **kw):
    def gpu(x):
        if x is None:
            return None
        base = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
        return base.copy_(x)

    d = {k: gpu(v) for k, v in t.items()}
    o = torch.full_like(d["y"], -7.0) if out else None
    r = torch.full_like(d["residual"], -7.0) if t["residual"] is not None else None
    cv.block_norm(d["y"], o, gate=d["gate"], post_weight=d["post_weight"], residual=d["residual"], residual_out=r,
                  channel_scale=d["channel_scale"], pre_weight=d["pre_weight"], **kw)
    torch.cuda.synchronize()
    return o, r


def bounds(t, out, res, dim, dtype, scale):
    """fp32: the sum of squares of n terms is off by at most n * 2^-24 relative, half of that in its root; the
    gate's exponential, its quotient, the root and the products add fewer than 16 roundings: a factor of
    (dim / 2 + 16) * 2^-24 of each value before it is rounded to its type.  The residual adds to |res|."""
    f = (dim / 2 + 16) * EPS32
    if res is None:
        tol = f * out.abs()
        return tol + (EPS16 * out.abs() if dtype == "bf16" else 0) + 1e-37, None
    base = t["residual"].double().abs()
    rt = f * ((res - t["residual"].double()).abs() + base)
    # out = r * inv * w: r's own error (relative to |r| + |res|), then the second norm's
    w = t["pre_weight"].double().abs() if t["pre_weight"] is not None else 1.0
    inv = 1 / torch.sqrt((res * res).mean(-1, keepdim=True) + 1e-6)
    ot = w * inv * rt + f * out.abs() + out.abs() * (inv * rt * inv * res.abs()).mean(-1, keepdim=True)
    rr = t["residual"].dtype == torch.bfloat16
    return (ot + (EPS16 * (out.abs() + ot) if dtype == "bf16" else 0) + 1e-37,
            rt + (EPS16 * (res.abs() + rt) if rr else 0) + 1e-37)


def check(cv, t, dim, dtype, scale=1.0, out=True, **kw):
    o, r = run(cv, t, dtype, out=out, scale=scale, **kw)
    ref = {k: v for k, v in t.items()}
    want, res = norm(scale=scale, **ref, **kw)
    ot, rt = bounds(t, want, res, dim, dtype, scale)
    if o is not None:
        assert_within(o, want, ot, "out")
    if r is not None:
        assert_within(r, res, rt, "residual_out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act,first", [("silu", False), ("sigmoid", False), ("silu", True)])
@pytest.mark.parametrize("rows,dim,group", [(1, 6144, 128), (5, 768, 64), (3, 96, 96), (700, 384, 128), (2, 40, 8),
                                            (4, 1000, 250), (3, 37, 37), (9, 6098, 6098), (2, 512, 512), (3, 7, 1),
                                            (33, 1536, 256), (2, 8192, 8192), (1, 16384, 16384), (1, 20000, 20000),
                                            (2, 2112, 1056), (1, 40000, 40000)])
def test_gated_norm(cuda_lib, rows, dim, group, act, first, dtype):
    t = make(rows, dim, dtype, seed=dim, group=group, gate=True)
    check(cuda_lib, t, group, dtype, gate_act=act, gate_first=first, group=group)


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,dim,group", [(1, 4096, 4096), (3, 4096, 0), (5, 1000, 1000), (2, 77, 77), (4, 512, 64),
                                            (3, 15, 5), (2, 8192, 8192), (2, 12288, 12288), (1, 24576, 24576),
                                            (2, 33, 0), (300, 256, 256)])
@pytest.mark.parametrize("gate", [False, True])
def test_residual_norm(cuda_lib, rows, dim, group, gate, dtype, res):
    t = make(rows, dim, dtype, seed=dim + rows, group=group, gate=gate, res=res, cs=rows % 2 == 1, pre=dim % 2 == 0)
    check(cuda_lib, t, dim, dtype, scale=0.3, group=group)


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,dim", [(2501, 520), (2500, 1024), (643, 64), (650, 63), (701, 200), (611, 300), (645, 517),
                                      (620, 1030), (610, 2047), (615, 4096), (3, 8199), (611, 8190)])
def test_many_rows(cuda_lib, rows, dim, dtype, res):
    """Enough rows that several share a block, or that later ones are prefetched."""
    t = make(rows, dim, dtype, seed=dim, group=dim, gate=True, res=res, cs=dim % 2 == 0, pre=True)
    check(cuda_lib, t, dim, dtype, scale=0.5, group=dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_residual_without_second_norm(cuda_lib, dtype):
    t = make(6, 512, dtype, seed=1, group=512, gate=True, res=dtype)
    check(cuda_lib, t, 512, dtype, scale=2.0, out=False, group=512)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [1, 3, 8])
def test_row_strides(cuda_lib, dtype, wide):
    t = make(5, 256, dtype, seed=wide, group=64, gate=True, wide=wide)
    check(cuda_lib, t, 64, dtype, group=64)
    t = make(5, 256, dtype, seed=wide, group=256, gate=True, res="f32", pre=True, wide=wide)
    check(cuda_lib, t, 256, dtype, group=256)


@pytest.mark.parametrize("dim,group", [(256, 64), (256, 256), (30000, 30000), (96, 8)])
def test_in_place(cuda_lib, dim, group):
    """out over y, residual_out over residual: the same bits as into buffers of their own."""
    t = make(9, dim, "bf16", seed=3, group=group, gate=True, res="f32", pre=True)
    want, res = run(cuda_lib, t, "bf16", group=group)
    y, r = t["y"].cuda(), t["residual"].cuda()
    cuda_lib.block_norm(y, y, gate=t["gate"].cuda(), group=group, post_weight=t["post_weight"].cuda(), residual=r,
                        residual_out=r, pre_weight=t["pre_weight"].cuda())
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(r, res)
    t["residual"] = t["pre_weight"] = None
    want, _ = run(cuda_lib, t, "bf16", group=group)
    y = t["y"].cuda()
    cuda_lib.block_norm(y, y, gate=t["gate"].cuda(), group=group, post_weight=t["post_weight"].cuda())
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_rows_of_zeros_infinities_and_nan(cuda_lib):
    """A row of zeros gives zeros (eps under the root); a bad row stays in its row, a bad group in its group."""
    t = make(4, 256, "f32", seed=4, group=64)
    t["y"][1] = 0
    t["y"][2, 70] = float("nan")
    o, _ = run(cuda_lib, t, "f32", group=64)
    assert float(o[1].abs().max()) == 0
    assert torch.isnan(o[2, 64:128]).all() and torch.isfinite(o[2, :64]).all() and torch.isfinite(o[2, 128:]).all()
    assert torch.isfinite(o[[0, 3]]).all()
    # very negative gates close, they do not overflow
    t = make(2, 128, "f32", seed=5, group=128, gate=True)
    t["gate"][:] = -200.0
    o, _ = run(cuda_lib, t, "f32", group=128)
    assert float(o.abs().max()) < 1e-30


def test_row_bits_do_not_depend_on_the_batch(cuda_lib):
    t = make(500, 6144, "bf16", seed=6, group=128, gate=True)
    o, _ = run(cuda_lib, t, "bf16", group=128)
    one = {k: (v[17:18] if v is not None and v.dim() == 2 else v) for k, v in t.items()}
    p, _ = run(cuda_lib, one, "bf16", group=128)
    assert torch.equal(o[17], p[0])


def test_no_rows_is_no_launch(cuda_lib):
    y = torch.zeros(0, 64, device="cuda")
    cuda_lib.block_norm(y, y.clone(), group=64)
