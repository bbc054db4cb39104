"""The operators that follow the conv of a hybrid layer, as a serving program calls them.

Three operators are measured:
  prefill  linear attention with a decay for each head over whole prompts, packed back to back
  step     the same recurrence over one new token, or over the draft tokens of a speculative verify,
           together with the deferred commit of the previous step's accepted drafts
  norm     the block norms: a gated norm over each head's channels, or the norm, gate and scaled
           residual after a block together with the norm before the next one

`run` computes each either in its plain form (elementary torch operations in fp32, rounded once) or,
where `own` is true, by the calls of spec_decode_verify_gb300.  `exact` gives the same results from the
definition in fp64, token by token.

Linear attention: for value head h, which reads the q|k head h * n_qk // n_heads,
    S_t = exp(g_t) S_{t-1} + b_t k_t v_t^T,      o_t = scale * S_t^T q_t + d v_t
with g the log decay, b the input gain and d the skip weight of the head.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases


def listed():
    return [
        # a short chat turn on its own: latency counts
        _prefill("prefill_1x33_h16x48_d128", "33", 16, 48, 128, 128, "bf16"),
        # the mixed prompts of the conv's prefill benchmark: dim 10240 = 16 q heads, 16 k heads and 48 v heads of 128
        _prefill("prefill_8x1k_7k_h16x48_d128", "2876,5823,3396,4746,3887,5385,3138,1571", 16, 48, 128, 128, "bf16",
                 init=True),
        # one long document on an eighth of the heads: few rows, so the length itself has to be split
        _prefill("prefill_1x32k_h2x6_d128", "32768", 2, 6, 128, 128, "bf16"),
        # many short prompts of a layer with one q|k group shared by all heads, narrow values, gain and skip
        _prefill("prefill_24x1_700_h1x64_k128_v64",
                 "1,700,37,128,129,255,64,511,3,320,90,633,18,257,412,77,200,149,583,31,366,5,474,111", 1, 64, 128, 64,
                 "bf16", init=True, gain=True, skip=True),
        # fp32 layer of the small configuration (dim 512: q 128, k 128, v 256, head_dim 64)
        _prefill("prefill_4x256_1k_h2x4_d64_f32", "256,1000,517,803", 2, 4, 64, 64, "f32", init=True, gain=True),
        # one new token of one sequence
        _step("decode_1x1_h16x48_d128", 1, 1, 16, 48, 128, 128, "bf16", update=True),
        # one new token of a batch, fp32
        _step("decode_64x1_h8x32_k64_v128_f32", 64, 1, 8, 32, 64, 128, "f32", update=True, gain=True),
        # the verify benchmark: 128 sequences of 8 drafts, 13 of them padded, with the previous step's commit
        _step("verify_128x8_pad13_h16x48_d128", 128, 8, 16, 48, 128, 128, "bf16", pad=13, prev=8),
        # packed drafts of 1..17 tokens, nothing to commit yet (the dim 8192 configuration: 2048 | 2048 | 4096)
        _step("verify_ragged_8x1_17_h16x32_d128", 8, 17, 16, 32, 128, 128, "bf16", ragged=True),
        # the gated norm of one decoded token, per head
        _norm("norm_gated_1x6144_g128", 1, 6144, "bf16", group=128, gate="silu"),
        # the same for the prompts above
        _norm("norm_gated_30822x6144_g128", 30822, 6144, "bf16", group=128, gate="silu"),
        # the end of a block and the start of the next one for a verify batch, fp32 residual stream
        _norm("norm_block_1023x4096_f32res", 1023, 4096, "bf16", group=4096, gate="sigmoid", residual="f32"),
    ]


def _prefill(name, lens, n_qk, n_heads, dk, dv, dtype, init=False, gain=False, skip=False):
    return {"name": name, "op": "prefill", "lens": lens, "n_qk": n_qk, "n_heads": n_heads, "dk": dk, "dv": dv,
            "dtype": dtype, "init": init, "gain": gain, "skip": skip}


def _step(name, n_seq, T, n_qk, n_heads, dk, dv, dtype, update=False, gain=False, skip=False, pad=0, prev=0, ragged=False):
    return {"name": name, "op": "step", "n_seq": n_seq, "T": T, "n_qk": n_qk, "n_heads": n_heads, "dk": dk, "dv": dv,
            "dtype": dtype, "update": update, "gain": gain, "skip": skip, "pad": pad, "prev": prev, "ragged": ragged}


def _norm(name, rows, dim, dtype, group=0, gate="", gate_first=False, residual="", pre=True):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "dtype": dtype, "group": group, "gate": gate,
            "gate_first": gate_first, "residual": residual, "pre": pre}


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["prefill", "step", "norm"])
    if op == "norm":
        rows = _log_int(rng, 1, 30000)
        residual = rng.choice(["", "same", "f32"])
        groups = rng.choice([1, 3, 8, 40]) if not residual else 1
        dim = _log_int(rng, 64, 8192) if groups == 1 else groups * rng.choice([64, 96, 128, 256])
        while rows * dim > 1.8e8:
            rows = rows // 2
        case = _norm("", rows, dim, rng.choice(["bf16", "bf16", "f32"]), group=dim // groups,
                     gate=rng.choice(["silu", "sigmoid"]) if not residual or rng.random() < 0.5 else "",
                     gate_first=rng.random() < 0.3, residual=residual, pre=rng.random() < 0.8)
    else:
        n_qk = rng.choice([1, 2, 4, 8])
        n_heads = n_qk * rng.choice([1, 2, 3, 4])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        dk, dv = rng.choice([64, 128, 128, rng.randrange(16, 129, 8)]), rng.choice([64, 128, 128, rng.randrange(16, 129, 8)])
        gain, skip = rng.random() < 0.5, rng.random() < 0.3
        if op == "prefill":
            n, top = _log_int(rng, 1, 32), _log_int(rng, 8, 16384 if dtype == "bf16" else 2048)
            lens = [rng.randint(1, top) for _ in range(n)]
            lens[rng.randrange(n)] = top
            while sum(lens) * n_heads > 500000:
                lens = [max(1, v // 2) for v in lens]
            case = _prefill("", ",".join(str(v) for v in lens), n_qk, n_heads, dk, dv, dtype, init=rng.random() < 0.5,
                            gain=gain, skip=skip)
        else:
            n, T = _log_int(rng, 1, 160), rng.choice([1, 1, rng.randint(2, 17), 4, 8])
            ragged = T > 1 and rng.random() < 0.4
            prev = 0 if T == 1 else rng.choice([0, T])
            case = _step("", n, T, n_qk, n_heads, dk, dv, dtype, update=T == 1, gain=gain, skip=skip,
                         pad=0 if ragged else n // 10, prev=prev, ragged=ragged)
    del case["name"]
    return case


# --------------------------------------------------------------------------------------- inputs


def _counts(case, seed):
    """Draft counts of the packed sequences, 1..T with T among them: a fixed spread, shuffled by the seed."""
    n, T = case["n_seq"], case["T"]
    c = [1 + (i * 7 + 3) % T for i in range(n)]
    c[0] = T
    k = seed % n
    return c[k:] + c[:k]


def _draft_total(case):
    return sum(_counts(case, 0)) if case["ragged"] else case["n_seq"] * case["T"]


def _tokens(g, lead, case, gain):
    """Views into one conv output row [q | k | v] per token, as the conv leaves them: q and k of unit norm
    per head, v after SiLU; log decays -a*dt with a in 1..16 per head and dt in 0.001..0.1; gains in (0, 1)."""
    nq, nh, dk, dv, dt = case["n_qk"], case["n_heads"], case["dk"], case["dv"], DTYPES[case["dtype"]]
    x = torch.randn(*lead, 2 * nq * dk + nh * dv, generator=g, device="cuda")
    qk = x[..., : 2 * nq * dk].view(*lead, 2 * nq, dk)
    qk /= qk.square().sum(-1, keepdim=True).add(1e-6).sqrt()
    v = x[..., 2 * nq * dk:]
    v *= torch.sigmoid(v)
    x = x.to(dt)
    q = x[..., : nq * dk].unflatten(-1, (nq, dk))
    k = x[..., nq * dk: 2 * nq * dk].unflatten(-1, (nq, dk))
    v = x[..., 2 * nq * dk:].unflatten(-1, (nh, dv))
    a = torch.exp(torch.rand(nh, generator=g, device="cuda") * math.log(16.0))
    dt_ = torch.exp(math.log(0.001) + torch.rand(*lead, nh, generator=g, device="cuda") * math.log(100.0))
    b = torch.sigmoid(torch.randn(*lead, nh, generator=g, device="cuda")) if gain else None
    return q, k, v, -a * dt_, b


def _cum(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        rows, dim = case["rows"], case["dim"]
        s["y"] = torch.randn(rows, dim, generator=g, device="cuda").to(dt)
        s["z"] = torch.randn(rows, dim, generator=g, device="cuda").to(dt) if case["gate"] else None
        s["w_post"] = (1 + 0.1 * torch.randn(case["group"], generator=g, device="cuda")).to(dt)
        s["out"] = torch.zeros(rows, dim, dtype=dt, device="cuda")
        s["res"] = None
        if case["residual"]:
            rdt = torch.float32 if case["residual"] == "f32" else dt
            s["res"] = torch.randn(rows, dim, generator=g, device="cuda").to(rdt)
            s["res_out"] = torch.zeros(rows, dim, dtype=rdt, device="cuda")
            s["w_pre"] = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(dt) if case["pre"] else None
            s["ch_scale"] = torch.rand(dim, generator=g, device="cuda").to(dt)
            if not case["pre"]:
                s["out"] = None
        return s
    nh, dk, dv = case["n_heads"], case["dk"], case["dv"]
    if case["op"] == "prefill":
        lens = [int(v) for v in case["lens"].split(",")]
        n, lead = len(lens), (sum(lens),)
        s["cu"], s["max_len"] = _cum(lens), max(lens)
        s["has_init"] = (torch.rand(n, generator=g, device="cuda") < 0.5).int() if case["init"] else \
            torch.zeros(n, dtype=torch.int32, device="cuda")
        pad = 0
    else:
        n, pad = case["n_seq"], case["pad"]
        lead = (_draft_total(case),) if case["ragged"] else (n, case["T"])
        s["cu"] = _cum(_counts(case, seed)) if case["ragged"] else None
    s["q"], s["k"], s["v"], s["g"], s["b"] = _tokens(g, lead, case, case["gain"])
    s["d"] = torch.rand(nh, generator=g, device="cuda") if case["skip"] else None
    s["scale"] = dk ** -0.5
    if case["op"] == "step" and case["prev"]:
        plead = lead if case["ragged"] else (n, case["prev"])
        _, s["pk"], s["pv"], s["pg"], s["pb"] = _tokens(g, plead, case, case["gain"])
        s["pcu"] = s["cu"]
        top = (s["cu"][1:] - s["cu"][:-1]) if case["ragged"] else torch.full((n,), case["prev"], device="cuda")
        s["accept"] = (1 + (torch.rand(n, generator=g, device="cuda") * top).floor()).clamp(max=top).int()
    slots = torch.randperm(n + n // 8, generator=g, device="cuda")
    s["state"] = torch.randn(n + n // 8, nh, dk, dv, generator=g, device="cuda") * 0.3
    s["slot"] = slots[:n].int()
    if pad:
        s["slot"][torch.randperm(n, generator=g, device="cuda")[:pad]] = -1
    s["out"] = torch.zeros(*lead, nh, dv, dtype=dt, device="cuda")
    return s


# ----------------------------------------------------------------------------------- plain forms


def _segments(x):
    """[..., L] -> [..., L, L]: sum of x over (j, i] for j <= i, -inf above the diagonal."""
    L = x.shape[-1]
    keep = torch.ones(L, L, dtype=torch.bool, device=x.device).tril(-1)
    s = torch.where(keep, x.unsqueeze(-1), 0.0).cumsum(-2)
    return s.masked_fill(~keep.logical_or(torch.eye(L, dtype=torch.bool, device=x.device)), -math.inf)


def _rows(t, at, ok):
    """Packed rows -> [n, L, ...] in fp32, zero where a sequence has none."""
    t = t[at]
    return torch.where(ok.view(*ok.shape, *[1] * (t.dim() - 2)), t.float(), 0.0)


def _chunked(q, k, v, g, b, S0, C):
    """[n, L, heads, d] in fp32, S0 [n, H, dk, dv] -> outputs [n, L, H, dv] (unscaled) and final states."""
    n, L, H, dv = v.shape
    heads = torch.arange(H, device=v.device) * k.shape[2] // H
    split = lambda t: t.transpose(1, 2).reshape(n, t.shape[2], L // C, C, *t.shape[3:])  # noqa: E731
    k, v, g, b = split(k)[:, heads], split(v), split(g), split(b)
    seg = _segments(g)
    decay_in = (seg[..., -1, :].exp() * b).unsqueeze(-1)
    local = (k * decay_in).transpose(-1, -2) @ v
    across = torch.cat([torch.zeros_like(g[..., :1, 0]), g.sum(-1)], -1)
    before = _segments(across).exp() @ torch.cat([S0.unsqueeze(2), local], 2).flatten(-2)
    before = before.unflatten(-1, (k.shape[-1], dv))
    if q is None:
        return None, before[:, :, -1]
    q = split(q)[:, heads]
    o = (q @ k.transpose(-1, -2) * seg.exp() * b.unsqueeze(-2)) @ v
    o = o + (q * g.cumsum(-1).exp().unsqueeze(-1)) @ before[:, :, :-1]
    return o.reshape(n, H, L, dv).transpose(1, 2), before[:, :, -1]


def _plain_prefill(s):
    cu, top, C = s["cu"].long(), s["max_len"], 64
    L = -(-top // C) * C
    pos = torch.arange(L, device="cuda")
    at = (cu[:-1, None] + pos).clamp(max=s["q"].shape[0] - 1)
    ok = pos < (cu[1:] - cu[:-1])[:, None]
    q, k, v, g = (_rows(s[name], at, ok) for name in "qkvg")
    b = _rows(s["b"], at, ok) if s["b"] is not None else ok[..., None].expand(g.shape).float()
    slot = s["slot"].long()
    S0 = torch.where(s["has_init"].bool()[:, None, None, None], s["state"][slot], 0.0)
    o, S = _chunked(q, k, v, g, b, S0, C)
    tok = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu, tok, right=True) - 1
    o = o[seq, tok - cu[seq]] * s["scale"]
    if s["d"] is not None:
        o = o + s["d"][:, None] * s["v"].float()
    s["out"].copy_(o)
    s["state"][slot] = S
    return s["out"], s["state"]


def _drafts(s, names, cu, T, counts):
    """The drafts as [n, T, ...] in fp32 rows, those at or past a sequence's count zero with no decay."""
    pos = torch.arange(T, device="cuda")
    ok = (pos < counts[:, None])
    at = (cu.long()[:-1, None] + pos).clamp(max=s[names[1]].shape[0] - 1) if cu is not None else None
    take = (lambda t: _rows(t, at, ok)) if at is not None else \
        (lambda t: torch.where(ok.view(*ok.shape, *[1] * (t.dim() - 2)), t.float(), 0.0))  # noqa: E731
    q, k, v, g, b = (take(s[x]) if x and s[x] is not None else None for x in names)
    return q, k, v, g, b if b is not None else ok[..., None].expand(g.shape).float()


def _plain_step(s):
    n, T = s["n_seq"], s["T"]
    live = s["slot"] >= 0
    slot = s["slot"].long().clamp(min=0)
    S = s["state"][slot]
    if s["prev"]:
        _, k, v, g, b = _drafts(s, (None, "pk", "pv", "pg", "pb"), s["pcu"], s["prev"], s["accept"])
        S = _chunked(None, k, v, g, b, S, s["prev"])[1]
        s["state"][slot[live]] = S[live]
    cu = s["cu"]
    counts = (cu[1:] - cu[:-1]) if cu is not None else torch.full((n,), T, device="cuda")
    q, k, v, g, b = _drafts(s, ("q", "k", "v", "g", "b"), cu, T, counts)
    o, S = _chunked(q, k, v, g, b, S, T)
    o = o * s["scale"]
    if s["d"] is not None:
        o = o + s["d"][:, None] * v
    if cu is not None:
        tok = torch.arange(s["q"].shape[0], device="cuda")
        seq = torch.searchsorted(cu.long(), tok, right=True) - 1
        s["out"].copy_(o[seq, tok - cu.long()[seq]])
    else:
        s["out"].copy_(torch.where(live[:, None, None, None], o, 0.0))
    if s["update"]:
        s["state"][slot[live]] = S[live]
    return s["out"], s["state"]


def _plain_norm(s):
    rows, dim, G = s["rows"], s["dim"], s["group"]
    u = s["y"].float()
    gate = None
    if s["z"] is not None:
        z = s["z"].float()
        gate = 1 / (1 + torch.exp(-z))
        gate = gate * z if s["gate"] == "silu" else gate
    if gate is not None and s["gate_first"]:
        u = u * gate
    u = u.view(rows, dim // G, G)
    u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + 1e-6) * s["w_post"].float()
    u = u.view(rows, dim)
    if gate is not None and not s["gate_first"]:
        u = u * gate
    if s["res"] is None:
        return u, None
    r = s["res"].float() + 0.5 * s["ch_scale"].float() * u
    if s["out"] is None:
        return None, r
    x = r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6)
    return (x * s["w_pre"].float() if s["w_pre"] is not None else x), r


def run(state):
    return _own(state) if own else _plain(state)


def _plain(s):
    if s["op"] == "prefill":
        return _plain_prefill(s)
    if s["op"] == "step":
        return _plain_step(s)
    out, res = _plain_norm(s)
    if out is not None:
        s["out"].copy_(out)
    if res is not None:
        s["res_out"].copy_(res)
        return s["out"], s["res_out"]
    return s["out"]


def _own(s):
    import spec_decode_verify_gb300 as cv
    if s["op"] == "prefill":
        cv.linattn_prefill(s["q"], s["k"], s["v"], s["g"], s["state"], s["out"], s["cu"], max_seqlen=s["max_len"],
                           gain=s["b"], skip=s["d"], scale=s["scale"], cache_idx=s["slot"],
                           has_initial_state=s["has_init"])
        return s["out"], s["state"]
    if s["op"] == "step":
        prev = cv.LinattnDrafts(s["pk"], s["pv"], s["pg"], s["accept"], gain=s["pb"], cu_draft=s["pcu"],
                                T=s["prev"]) if s["prev"] else None
        cv.linattn_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["out"], gain=s["b"], skip=s["d"],
                        scale=s["scale"], update_state=s["update"], prev=prev, cache_idx=s["slot"], cu_draft=s["cu"],
                        T=s["T"])
        return s["out"], s["state"]
    if s["res"] is None:
        cv.block_norm(s["y"], s["out"], gate=s["z"], gate_act=s["gate"] or None, gate_first=s["gate_first"],
                      group=s["group"], post_weight=s["w_post"], eps=1e-6)
        return s["out"]
    cv.block_norm(s["y"], s["out"], gate=s["z"], gate_act=s["gate"] or None, gate_first=s["gate_first"],
                  group=s["group"], post_weight=s["w_post"], residual=s["res"], residual_out=s["res_out"], scale=0.5,
                  channel_scale=s["ch_scale"], pre_weight=s["w_pre"], eps=1e-6)
    return s["out"], s["res_out"]


# ------------------------------------------------------------------------------------------ work


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, r = case["rows"] * case["dim"], 4 if case["residual"] == "f32" else e
        per = (2 + bool(case["gate"])) * e
        if case["residual"]:
            per = (1 + bool(case["gate"]) + case["pre"]) * e + 2 * r
        return {"bytes": n * per, "flops": n * (14 if case["residual"] else 8)}
    nq, nh, dk, dv = case["n_qk"], case["n_heads"], case["dk"], case["dv"]
    kv = (nq * dk + nh * dv) * e + nh * (8 if case["gain"] else 4)
    token = kv + (nq * dk + nh * dv) * e
    S = nh * dk * dv * 4
    if case["op"] == "prefill":
        lens = [int(v) for v in case["lens"].split(",")]
        return {"bytes": sum(lens) * token + len(lens) * S * (1.5 if case["init"] else 1),
                "flops": sum(lens) * nh * 4 * dk * dv}
    live = case["n_seq"] - case["pad"]
    new = _draft_total(case) * live / case["n_seq"]
    old = (new + live) / 2 if case["prev"] else 0  # accepted, on average
    write = case["update"] or case["prev"]
    return {"bytes": new * token + old * kv + live * S * (2 if write else 1),
            "flops": nh * dk * dv * (new * 4 + old * 2)}


# ----------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        out, res = _exact_norm(s)
        return out if s["res"] is None else (out, res)

    def recur(S, q, k, v, g, b, d, scale, counts, heads):
        """The definition token by token in fp64: [n, T, heads, d] rows, S [n, H, dk, dv]; sequence i stops after
        counts[i] tokens.  Outputs [n, T, H, dv] (None without q) and the states."""
        o = []
        for t in range(k.shape[1]):
            on = (t < counts)[:, None, None, None]
            kt, vt = k[:, t][:, heads].double(), v[:, t].double()
            bt = b[:, t].double() if b is not None else torch.ones_like(g[:, t], dtype=torch.float64)
            new = torch.exp(g[:, t].double())[..., None, None] * S + (bt[..., None] * kt)[..., None] * vt[:, :, None]
            S = torch.where(on, new, S)
            if q is not None:
                y = scale * (q[:, t][:, heads].double()[..., None, :] @ S).squeeze(-2)
                o.append(y + d.double()[:, None] * vt if d is not None else y)
        return (torch.stack(o, 1) if o else None), S

    heads = torch.arange(case["n_heads"], device="cuda") * case["n_qk"] // case["n_heads"]
    state, out = s["state"].double(), torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    live = (s["slot"] >= 0).nonzero().flatten()
    slot = s["slot"][live].long()
    S = state[slot]

    def rows(t, cu, T):
        if t is None:
            return None
        if cu is None:
            return t[live]
        lo = cu[:-1].long()[live]
        return t[(lo[:, None] + torch.arange(T, device="cuda")).clamp(max=t.shape[0] - 1)]

    if case["op"] == "prefill":
        S = S * s["has_init"][live].double()[:, None, None, None]
        T = s["max_len"]
    else:
        T = case["T"]
        if case["prev"]:
            pk, pv, pg, pb = (rows(s[x], s["pcu"], case["prev"]) for x in ("pk", "pv", "pg", "pb"))
            S = recur(S, None, pk, pv, pg, pb, None, 0.0, s["accept"][live], heads)[1]
            state[slot] = S
    cu = s["cu"]
    counts = (cu[1:] - cu[:-1])[live] if cu is not None else torch.full((len(live),), T, device="cuda")
    q, k, v, g, b = (rows(s[x], cu, T) for x in ("q", "k", "v", "g", "b"))
    o, S = recur(S, q, k, v, g, b, s["d"], s["scale"], counts, heads)
    if cu is None:
        out[live] = o
    else:
        ok = torch.arange(T, device="cuda") < counts[:, None]
        out[(cu[:-1].long()[live][:, None] + torch.arange(T, device="cuda"))[ok]] = o[ok]
    if case["op"] == "prefill" or case["update"]:
        state[slot] = S
    return out, state


def _exact_norm(s):
    """The norms by group sums in fp64: mean square over each group, then scale, gate and residual."""
    y = s["y"].double()
    gate = torch.ones_like(y)
    if s["z"] is not None:
        gate = torch.sigmoid(s["z"].double())
        if s["gate"] == "silu":
            gate = gate * s["z"].double()
    a = y * gate if s["gate_first"] else y
    inv = (a.pow(2).unflatten(-1, (-1, s["group"])).sum(-1) / s["group"] + 1e-6).pow(-0.5)
    u = a * inv.repeat_interleave(s["group"], -1) * s["w_post"].double().repeat(s["dim"] // s["group"])
    if not s["gate_first"]:
        u = u * gate
    if s["res"] is None:
        return u, None
    r = s["res"].double() + u * (s["ch_scale"].double() * 0.5)
    if s["out"] is None:
        return None, r
    inv = (r.pow(2).sum(-1, keepdim=True) / s["dim"] + 1e-6).pow(-0.5)
    return r * inv * (s["w_pre"].double() if s["w_pre"] is not None else 1.0), r
