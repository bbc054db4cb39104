"""Norms of query and key heads with the rotation, and the cache rows they write, against 64 bits."""
from __future__ import annotations

import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def angles(n, rot):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def close(got, want, x, weight, dtype):
    """fp32 arithmetic, rounded once: the norm's factor and the products are off by at most (d + 8) 2^-24, and a rotated value by
    that of the two channels it is made of, whose size is at most that of the row's largest scaled channel times 2^0.5."""
    d = x.shape[-1]
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    top = want.abs().amax(-1, keepdim=True) * 2 ** 0.5
    return bool(((got.double() - want).abs() <= half * want.abs() * 1.01 + (d + 8) * 2.0 ** -24 * top).all())


CASES = [  # H, n_kv, d, rot, pairs, norm, weight
    (4, 2, 128, 128, False, True, True), (3, 1, 64, 32, True, True, True), (8, 2, 256, 64, False, True, False), (2, 2, 96, 96, True, True, True),
    (5, 1, 80, 16, False, False, False), (2, 1, 48, 0, False, True, True), (1, 1, 20, 14, False, True, True), (2, 1, 33, 32, True, True, True),
    (0, 2, 64, 64, False, True, True), (2, 0, 64, 64, False, True, True), (1, 1, 1, 0, False, True, True), (2, 2, 250, 250, False, False, False)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,n_kv,d,rot,pairs,norm,weight", CASES)
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_forms(cuda_lib, H, n_kv, d, rot, pairs, norm, weight, packed, paged, dtype):
    cv = cuda_lib
    paged = paged and n_kv > 0
    g = torch.Generator().manual_seed(H * d + rot)
    counts = [5, 0, 17, 1] if packed else [3] * 4
    lens = [0, 9, 30, 7]
    n, T, page = 4, max(counts), 8
    lead = (sum(counts),) if packed else (n, 3)
    x = torch.randn(*lead, (H + 2 * n_kv) * d + 16, generator=g).to(dtype).cuda()
    q = x[..., :H * d].unflatten(-1, (H, d)) if H else torch.empty(*lead, 0, d, dtype=dtype, device="cuda")
    k = x[..., H * d:(H + n_kv) * d].unflatten(-1, (n_kv, d)) if n_kv else None
    v = x[..., (H + n_kv) * d:(H + 2 * n_kv) * d].unflatten(-1, (n_kv, d)) if n_kv else None
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() if weight else None for _ in range(2))
    cs = angles(60, rot).cuda() if rot else None
    slots = torch.tensor([2, 0, -1, 3], dtype=torch.int32)
    cu = torch.tensor([0] + counts).cumsum(0).int() if packed else None
    seq = torch.repeat_interleave(torch.arange(n), torch.tensor(counts))
    at = torch.cat([torch.arange(c) for c in counts])
    pos = (torch.tensor(lens)[seq] + at)
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    k_out = torch.full(k.shape, 7.0, dtype=dtype, device="cuda") if k is not None else None
    table = torch.randperm(4 * 7, generator=g).int().view(4, 7)
    cache = None
    if paged:
        cache = cv.PagedCache(torch.full((28, page, n_kv, d), 7.0, dtype=dtype, device="cuda"),
                              torch.full((28, page, n_kv, d), 7.0, dtype=dtype, device="cuda"), table.cuda())
    err = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    cv.qk_norm_rope(q, k, out, k_out=k_out if not paged or packed else None, v=v if paged else None, cos_sin=cs, q_weight=wq,
                    k_weight=wk, norm=norm, pairs=pairs, cache=cache, cache_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                    cu_seqlens=cu.cuda() if packed else None, max_seqlen=T, cache_idx=slots.cuda(), err=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0] * n
    live = slots[seq] >= 0
    cos, sin = (cs.cpu()[pos][:, :rot // 2], cs.cpu()[pos][:, rot // 2:]) if rot else (torch.zeros(len(pos), 0), torch.zeros(len(pos), 0))
    flat = lambda t: t.cpu().reshape(-1, *t.shape[-2:])  # noqa: E731
    for src, w, got in ((q, wq, out), (k, wk, k_out if not paged or packed else None)):
        if src is None or got is None or src.shape[-2] == 0:
            continue
        want = ref.norm_rope(flat(src), w.cpu() if w is not None else None, cos, sin, pairs, norm, 1e-6)
        assert close(flat(got)[live], want[live], src, w, dtype)
        assert bool((flat(got)[~live] == 7).all())
    if paged:
        want = ref.norm_rope(flat(k), wk.cpu() if wk is not None else None, cos, sin, pairs, norm, 1e-6)
        touched = torch.zeros(28, page, dtype=torch.bool)
        for i in range(len(pos)):
            if live[i]:
                pg, r = int(table[slots[seq[i]], int(pos[i]) // page]), int(pos[i]) % page
                touched[pg, r] = True
                assert close(cache.k[pg, r].cpu(), want[i], k, wk, dtype)
                assert torch.equal(cache.v[pg, r].cpu(), flat(v)[i])
        assert bool((cache.k.cpu()[~touched] == 7).all()) and bool((cache.v.cpu()[~touched] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 20])
def test_in_place_and_far_positions(cuda_lib, d, dtype):
    cv = cuda_lib
    g = torch.Generator().manual_seed(0)
    q, k = torch.randn(2, 3, 4, d, generator=g).to(dtype), torch.randn(2, 3, 1, d, generator=g).to(dtype)
    n = 100_000
    cs = angles(n, d)
    pos = torch.randint(n, (2, 3), generator=g).int()
    pos[0, 0] = n - 1
    a, b = q.cuda(), k.cuda()
    cv.qk_norm_rope(a, b, a, k_out=b, cos_sin=cs.cuda(), positions=pos.cuda())
    for got, x in ((a, q), (b, k)):
        z = cs[pos.long()]
        want = ref.norm_rope(x, None, z[..., :d // 2], z[..., d // 2:], False, True, 1e-6)
        assert close(got.cpu(), want, x, None, dtype)


def test_zero_rows_infinities_and_nan(cuda_lib):
    cv = cuda_lib
    q = torch.randn(1, 4, 1, 64).cuda()
    q[0, 0], q[0, 1, 0, 3], q[0, 2, 0, 5] = 0, float("inf"), float("nan")
    out = torch.empty_like(q)
    cv.qk_norm_rope(q, None, out)
    assert bool((out[0, 0] == 0).all()) and bool(torch.isnan(out[0, 2]).all())
    assert bool(torch.isnan(out[0, 1, 0, 3])) and bool((out[0, 1, 0, :3] == 0).all())
    assert bool(torch.isfinite(out[0, 3]).all())


@pytest.mark.parametrize("d", [64, 20])
def test_flags(cuda_lib, d):
    """Tokens whose page or position is not there are left out; a sequence of a bad slot, span or length as a whole."""
    cv = cuda_lib
    n, T, page = 6, 4, 8
    q = torch.randn(n, T, 2, d, device="cuda")
    k = torch.randn(n, T, 1, d, device="cuda")
    table = torch.arange(n * 3, dtype=torch.int32).view(n, 3)
    table[2, 1] = 99
    cache = cv.PagedCache(torch.full((n * 3, page, 1, d), 7.0, device="cuda"), torch.full((n * 3, page, 1, d), 7.0, device="cuda"),
                          table.cuda())
    lens = torch.tensor([0, 0, 6, 21, -1, 0], dtype=torch.int32).cuda()
    slots = torch.tensor([0, n, 2, 3, 4, 5], dtype=torch.int32).cuda()
    pos = torch.arange(T, dtype=torch.int32).expand(n, T).contiguous()
    pos[5, 2], pos[0, 3] = 50, 49
    out, err = torch.full_like(q, 7.0), torch.full((n,), -7, dtype=torch.int32, device="cuda")
    cv.qk_norm_rope(q, k, out, v=k.clone(), cos_sin=angles(50, d).cuda(), positions=pos.cuda(), cache=cache, cache_len=lens, cache_idx=slots,
                    err=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 1, 128, 64, 64, 2048]
    left = (out == 7).all(-1).all(-1).tolist()
    assert left == [[False] * 4, [True] * 4, [False, False, True, True], [True] * 4, [True] * 4, [False, False, True, False]]
    assert bool((cache.k[table[5, 0], 2] == 7).all()) and bool((cache.k[table[5, 0], 3] != 7).all())


def test_bad_spans(cuda_lib):
    cv = cuda_lib
    q = torch.randn(10, 1, 32, device="cuda")
    out, err = torch.full_like(q, 7.0), torch.full((3,), -7, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3, 8, 9], dtype=torch.int32, device="cuda")
    cv.qk_norm_rope(q, None, out, cu_seqlens=cu, max_seqlen=4, err=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 16, 0]
    assert (out == 7).all(-1).flatten().tolist() == [False] * 3 + [True] * 5 + [False] + [True]


def test_long_prompts_of_many_heads(cuda_lib):
    cv = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(0)
    lens = [1500, 1, 700]
    q, k = (torch.randn(sum(lens), h, 128, generator=g, device="cuda").bfloat16() for h in (16, 4))
    cs = angles(1500, 128).cuda()
    out, k_out = torch.empty_like(q), torch.empty_like(k)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    cv.qk_norm_rope(q, k, out, k_out=k_out, cos_sin=cs, cache_len=torch.zeros(3, dtype=torch.int32, device="cuda"), cu_seqlens=cu,
                    max_seqlen=1500)
    pos = torch.cat([torch.arange(c) for c in lens])
    for got, x in ((out, q), (k_out, k)):
        want = ref.norm_rope(x.cpu(), None, cs.cpu()[pos][:, :64], cs.cpu()[pos][:, 64:], False, True, 1e-6)
        assert close(got.cpu(), want, x, None, BF)
