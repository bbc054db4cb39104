"""Plain fp64 forms of the operators beside the conv, token by token and row by row (CPU tensors)."""
from __future__ import annotations

import torch

EPS32 = 2.0 ** -24  # half a unit in the last place of fp32, relative
EPS16 = 2.0 ** -8   # the same of bf16 (8 significant bits)


def linattn(S, q, k, v, g, b=None, d=None, scale=1.0):
    """One sequence: S [H, dk, dv], q, k [T, Hq, dk] (q may be None), v [T, H, dv], g, b [T, H], d [H].

    Returns outputs [T, H, dv] (None without q), the final state, and for both the same sums over absolute
    values (what a rounding error is relative to), all fp64."""
    H = v.shape[1]
    heads = torch.arange(H) * k.shape[1] // H
    S, M, out, mag = S.double(), S.double().abs(), [], []
    for t in range(k.shape[0]):
        a = torch.exp(g[t].double())[:, None, None]
        w = b[t].double()[:, None] if b is not None else torch.ones(H, 1, dtype=torch.float64)
        kv = (w * k[t].double()[heads])[:, :, None] * v[t].double()[:, None, :]
        S, M = a * S + kv, a * M + kv.abs()
        if q is not None:
            qt = q[t].double()[heads][:, :, None]
            o, m = scale * (qt * S).sum(1), abs(scale) * (qt.abs() * M).sum(1)
            if d is not None:
                o, m = o + d.double()[:, None] * v[t].double(), m + (d.double()[:, None] * v[t].double()).abs()
            out.append(o)
            mag.append(m)
    if q is None:
        return None, S, None, M
    if not out:
        z = torch.zeros(0, H, v.shape[2], dtype=torch.float64)
        return z, S, z, M
    return torch.stack(out), S, torch.stack(mag), M


def linattn_bounds(mag, out, dk, n, dtype, chunked):
    """Error bound of each output or state element (derived, not fitted).

    fp32 arithmetic: a term passes at most dk + n additions, n decays of at most 4 roundings each (the
    exponential's 2 ulp and the product) and a few more products, each off by at most 2^-24 of the sum of
    absolute values.  The chunked kernel (bf16 only) rounds the decayed products q.k and the state it reads
    to bf16 (2^-8 relative each, so at most 2^-8 of the sum), and writes the weighted keys of the
    state update as a high and a low bf16 part (2^-16 relative).  out: None for a state (fp32), else the
    outputs, rounded once to dtype."""
    tol = (dk + 8 * n + 32) * EPS32 * mag
    if chunked:
        tol = tol + (2.0 ** -16 if out is None else EPS16) * mag
    if out is not None and dtype == torch.bfloat16:
        tol = tol + EPS16 * (out.abs() + tol)
    return tol + 1e-37


def assert_within(got, want, tol, what):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} vs {tuple(want.shape)}"
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN positions differ"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~nan & ~inf
    off = (got - want).abs()[ok]
    lim = tol.expand_as(want)[ok]
    if off.numel() and bool((off > lim).any()):
        i = int((off - lim).argmax())
        raise AssertionError(f"{what}: {int((off > lim).sum())} of {off.numel()} beyond the bound; worst got "
                             f"{float(got[ok][i])} want {float(want[ok][i])} bound {float(lim[i])}")


def norm(y, *, gate=None, gate_act="silu", gate_first=False, group=0, post_weight=None, residual=None, scale=1.0,
         channel_scale=None, pre_weight=None, eps=1e-6):
    """(out, residual_out) of the block norm in fp64; the second None without a residual."""
    a = y.double()
    z = None
    if gate is not None:
        z = torch.sigmoid(gate.double())
        z = z * gate.double() if gate_act == "silu" else z
    if z is not None and gate_first:
        a = a * z
    if group:
        x = a.reshape(y.shape[0], -1, group)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if post_weight is not None:
            x = x * post_weight.double()
        a = x.reshape(y.shape)
    if z is not None and not gate_first:
        a = a * z
    if residual is None:
        return a, None
    r = residual.double() + scale * a * (channel_scale.double() if channel_scale is not None else 1.0)
    x = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return (x * pre_weight.double() if pre_weight is not None else x), r
