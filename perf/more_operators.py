"""The operators of a hybrid model's attention layers under speculative decoding, as a serving program calls them.

Four operators are measured:
  attend   attention of drafted tokens (a chain or a tree of them) over a paged cache
  sample   verification of drafted tokens against the target's probabilities, from given random numbers
  rope     norms of queries and keys for each head with the position rotation, written into the cache's pages
  pages    the cache's pages: compacting the accepted path, and forking, growing and freeing sequences

`run` computes each either in its plain form (elementary torch operations in fp32, rounded once; the sums of the
sampling in fp64) or, where `own` is true, by the calls of spec_decode_verify_gb300.  `exact` gives the same
results from the definitions in 64 bits, sequence by sequence.

Draft token t of a sequence has a parent in [-1, t); without parents token t follows token t-1.  Token 0 is the
token sampled by the last step.  Its K and V stand in the cache at position cache_len + t.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one decoded token of one chat: latency counts
        _attend("attend_1x1_ctx700_h16x2_d128", 1, 1, 700, 16, 2, 128, 16, "bf16"),
        # the verify benchmark's batch: 128 sequences of 8 drafts in a tree, 13 of them padded
        _attend("attend_128x8_tree_ctx8k_h32x4_d128", 128, 8, 8000, 32, 4, 128, 16, "bf16", tree=True, pad=13),
        # one long document with 17 drafts: few rows, so the length itself has to be split; more rows than one tile
        _attend("attend_1x17_ctx100k_h64x8_d128", 1, 17, 100001, 64, 8, 128, 64, "bf16"),
        # packed trees of 1..17 drafts of the small fp32 configuration's heads of 64
        _attend("attend_ragged_8x1_17_tree_ctx1k_h8x4_d64_f32", 8, 17, 1100, 8, 4, 64, 32, "f32", tree=True, ragged=True),
        # one sequence with 3 drafts and their probabilities
        _sample("sample_1x4_v32000_q", 1, 4, 32000, "f32", q=True),
        # the verify benchmark's batch over a large vocabulary
        _sample("sample_128x8_pad13_v128000_q", 128, 8, 128000, "f32", q=True, pad=13),
        # packed trees of drafts without probabilities (looked up in the text), bf16 probabilities
        _sample("sample_ragged_64x1_16_tree_v50257_bf16", 64, 16, 50257, "bf16", tree=True, ragged=True),
        # one decoded token
        _rope("rope_1x1_h16x2_d128", 1, 1, 16, 2, 128, 128, "bf16"),
        # the mixed prompts of the conv's prefill benchmark
        _rope("rope_8x1k_7k_h32x8_d128", 8, 7000, 32, 8, 128, 128, "bf16", ragged=True),
        # the verify benchmark's batch, a quarter of each wide head rotated, neighbouring channels as pairs
        _rope("rope_128x8_pad13_h16x2_d256_r64_pairs", 128, 8, 16, 2, 256, 64, "bf16", pad=13, pairs=True),
        # the accepted paths of 128 trees, moved to their places in 16 layers
        _compact("compact_128x16_l16_h8_d128", 128, 16, 16, 8, 128, 16, "bf16", pad=13),
        # 64 continuations of 4 prompts: the old ones freed, new ones forked and grown by 8 tokens
        _fork("fork_64of4_ctx2k_l4_h8_d128", 64, 4, 2005, 8, 4, 8, 128, 16, "bf16"),
    ]


def _attend(name, n_seq, T, ctx, n_heads, n_kv, d, page, dtype, tree=False, ragged=False, pad=0):
    return {"name": name, "op": "attend", "n_seq": n_seq, "T": T, "ctx": ctx, "n_heads": n_heads, "n_kv": n_kv, "d": d,
            "page": page, "dtype": dtype, "tree": tree, "ragged": ragged, "pad": pad}


def _sample(name, n_seq, T, vocab, dtype, q=False, tree=False, ragged=False, pad=0):
    return {"name": name, "op": "sample", "n_seq": n_seq, "T": T, "vocab": vocab, "dtype": dtype, "q": q, "tree": tree,
            "ragged": ragged, "pad": pad}


def _rope(name, n_seq, T, n_heads, n_kv, d, rot, dtype, ragged=False, pad=0, pairs=False, page=16):
    return {"name": name, "op": "rope", "n_seq": n_seq, "T": T, "n_heads": n_heads, "n_kv": n_kv, "d": d, "rot": rot,
            "dtype": dtype, "ragged": ragged, "pad": pad, "pairs": pairs, "page": page}


def _compact(name, n_seq, T, layers, n_kv, d, page, dtype, pad=0):
    return {"name": name, "op": "compact", "n_seq": n_seq, "T": T, "layers": layers, "n_kv": n_kv, "d": d, "page": page,
            "dtype": dtype, "pad": pad}


def _fork(name, n_dst, n_src, ctx, grow, layers, n_kv, d, page, dtype):
    return {"name": name, "op": "fork", "n_dst": n_dst, "n_src": n_src, "ctx": ctx, "grow": grow, "layers": layers,
            "n_kv": n_kv, "d": d, "page": page, "dtype": dtype}


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "sample", "rope", "compact", "fork"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    n_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    d = rng.choice([64, 128, 128, 256, rng.randrange(16, 129, 16)])
    page = rng.choice([16, 16, 32, 64, 128])
    n, T = _log_int(rng, 1, 128), rng.choice([1, 1, 4, 8, rng.randint(2, 24)])
    ragged = T > 1 and rng.random() < 0.3
    pad = 0 if ragged else n // 10
    if op == "attend":
        ctx = _log_int(rng, 1, 32000)
        while n * ctx * n_kv * d > 1.2e8 or n * ctx * n_kv * group * T > 2.5e8 or (
                dtype == "f32" and n * ctx * n_kv * group * T * d > 3e9):
            ctx, n = ctx // 2 + 1, n // 2 + 1
            pad = 0 if ragged else n // 10
        case = _attend("", n, T, ctx, n_kv * group, n_kv, d, page, dtype, tree=rng.random() < 0.5, ragged=ragged, pad=pad)
    elif op == "sample":
        vocab, T = _log_int(rng, 500, 150000), max(T, 2)
        q = rng.random() < 0.5
        while n * T * vocab > 1.3e8:
            n = n // 2
            pad = 0 if ragged else n // 10
        case = _sample("", n, T, vocab, dtype, q=q, tree=not q and rng.random() < 0.6, ragged=ragged, pad=pad)
    elif op == "rope":
        if rng.random() < 0.5:
            T, ragged, pad = _log_int(rng, 30, 8000), True, 0
        while n * T * n_kv * (group + 2) * d > 1.8e8:
            n, pad = n // 2, 0
        pairs = rng.random() < 0.4
        case = _rope("", n, T, n_kv * group, n_kv, d, rng.choice([d, d, d // 2 // 8 * 8]), dtype, ragged=ragged, pad=pad,
                     pairs=pairs, page=page)
    elif op == "compact":
        T, layers = max(T, 2), _log_int(rng, 1, 16)
        while n * (40 + T) * layers * n_kv * d > 3e8:
            layers = layers // 2 + (layers == 1)
            n = n // 2 + 1 if layers == 1 else n
        case = _compact("", n, T, layers, n_kv, d, page, dtype, pad=n // 10)
    else:
        n_src, layers = max(1, n // rng.choice([4, 8, 16])), _log_int(rng, 1, 8)
        ctx = _log_int(rng, 1, 3000)
        while (n_src * ctx + n * 6 * page) * layers * n_kv * d > 3e8:
            ctx, layers, n = ctx // 2 + 1, layers // 2 + (layers == 1), n // 2 + (n == 1)
            n_src = min(n_src, n)
        case = _fork("", n, n_src, ctx, rng.randint(1, 40), layers, n_kv, d, page, dtype)
    del case["name"]
    return case


# --------------------------------------------------------------------------------------- inputs


def _spread(n, top, seed, low=0):
    """n lengths in low..top with top among them: a fixed spread, rotated by the seed."""
    c = [low + (i * 7919 + 13) % (top - low + 1) for i in range(n)]
    c[0] = top
    k = seed % n
    return c[k:] + c[:k]


def _counts(case, seed):
    n, T = case["n_seq"], case["T"]
    return _spread(n, T, seed, 1) if case["ragged"] else [T] * n


def _ints(v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


def _cum(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


def _table(g, need, page, extra=0):
    """A page table whose row s holds pages for need[s] tokens, the pages in random order; entries past them are -1."""
    pages = [-(-v // page) for v in need]
    total = sum(pages)
    order = torch.randperm(total + extra, generator=g, device="cuda").int()
    table = torch.full((len(need), max(max(pages), 1)), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(table.shape[1], device="cuda")
    table[col < _ints(pages)[:, None]] = order[:total]
    return table, total + extra


def _slots(g, n, rows, pad):
    slot = torch.randperm(rows, generator=g, device="cuda")[:n].int()
    if pad:
        slot[torch.randperm(n, generator=g, device="cuda")[:pad]] = -1
    return slot


def _parents(g, n, T, reach):
    """Random trees: token t's parent is one of the `reach` tokens before it; token 0 is the root."""
    t = torch.arange(T, device="cuda")
    back = 1 + (torch.rand(n, T, generator=g, device="cuda") * reach).floor().int()
    return torch.maximum(t - back, torch.zeros_like(t)).where(t > 0, -1).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"attend": _prepare_attend, "sample": _prepare_sample, "rope": _prepare_rope, "compact": _prepare_compact,
            "fork": _prepare_fork}[case["op"]](dict(case), g, seed)


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=DTYPES[dtype])


def _prepare_attend(s, g, seed):
    n, T, kv, d, page = s["n_seq"], s["T"], s["n_kv"], s["d"], s["page"]
    counts, lens = _counts(s, seed), _spread(n, s["ctx"], seed)
    s["counts"], s["top"] = _ints(counts), s["ctx"] + T
    table, n_pages = _table(g, [v + c for v, c in zip(lens, counts)], page, extra=3)
    s["slot"] = _slots(g, n, n, s["pad"])
    s["table"] = torch.empty_like(table)
    on = s["slot"].long().clamp(min=0)
    s["table"].fill_(-1)
    s["table"][on[s["slot"] >= 0]] = table[s["slot"] >= 0]
    s["len"] = _ints(lens)
    s["k"] = _randn(g, n_pages, page, kv, d, dtype=s["dtype"])
    s["v"] = _randn(g, n_pages, page, kv, d, dtype=s["dtype"])
    s["cu"] = _cum(counts) if s["ragged"] else None
    lead = (sum(counts),) if s["ragged"] else (n, T)
    s["q"] = _randn(g, *lead, s["n_heads"], d, dtype=s["dtype"])
    parent = _parents(g, n, T, 3) if s["tree"] else None
    s["all_parents"] = parent
    s["parent"] = _pack(parent, counts) if s["ragged"] and s["tree"] else parent
    s["out"] = torch.zeros_like(s["q"])
    _hold(s)
    return s


def _hold(s, **pool):
    """The library's handle of the cache's tensors, which a program makes once for each layer."""
    if own:
        import spec_decode_verify_gb300 as cv
        s["cache"] = cv.PagedCache(s["k"], s["v"], s["table"], **pool)


def _pack(t, counts):
    return torch.cat([t[i, :c] for i, c in enumerate(counts)])


def _prepare_sample(s, g, seed):
    """Target rows as a softmax leaves them (a few likely tokens, a long tail); drafts from a distribution near the
    target's, or without probabilities from the target's own likely tokens."""
    n, T, V, dt = s["n_seq"], s["T"], s["vocab"], DTYPES[s["dtype"]]
    counts = _counts(s, seed)
    parent = _parents(g, n, T, 3) if s["tree"] else None
    logits = torch.randn(n, T, V, generator=g, device="cuda") * 4
    p = torch.softmax(logits, -1).to(dt)
    q = None
    if s["q"]:
        logits += torch.randn(n, T, V, generator=g, device="cuda")
        q = torch.softmax(logits, -1).to(dt)
    # token t is drawn for the place after its parent
    up = parent.long().clamp(min=0) if parent is not None else (torch.arange(T, device="cuda") - 1).clamp(min=0).expand(n, T)
    rows = torch.arange(n, device="cuda")[:, None].expand(n, T)
    tok = torch.empty(n, T, dtype=torch.int32, device="cuda")
    for t in range(T):
        of = q if q is not None else p
        tok[:, t] = torch.multinomial(of[rows[:, t], up[:, t]].float(), 1, generator=g)[:, 0].int()
    if q is not None:  # row t: the distribution that token t was drawn from
        q = torch.cat([q[:, :1], q[:, :-1]], 1).contiguous()
    u = torch.rand(n, T + 1, generator=g, device="cuda")
    s["cu"] = _cum(counts) if s["ragged"] else None
    s["counts"], s["all_parents"] = _ints(counts), parent
    if s["ragged"]:
        p, tok = _pack(p, counts), _pack(tok, counts)
        q = _pack(q, counts) if q is not None else None
        parent = _pack(parent, counts) if parent is not None else None
    s["p"], s["qp"], s["tok"], s["parent"], s["u"] = p, q, tok, parent, u
    s["slot"] = _slots(g, n, n, s["pad"])
    s["accept"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["node"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["new"] = torch.zeros(n, T, dtype=torch.int32, device="cuda")
    s["path"] = torch.zeros(n, T, dtype=torch.int32, device="cuda")
    return s


def _prepare_rope(s, g, seed):
    n, T, kv, d, H, page = s["n_seq"], s["T"], s["n_kv"], s["d"], s["n_heads"], s["page"]
    counts = _counts(s, seed)
    prompt = s["ragged"]
    lens = [0] * n if prompt else _spread(n, 40, seed)
    far = 0 if prompt else 30000  # positions of decoded tokens; the cache here holds only the last pages
    top = far + 40 + T
    half = s["rot"] // 2
    angle = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * \
        1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(half, 1))
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    table, n_pages = _table(g, [v + c for v, c in zip(lens, counts)], page, extra=3)
    s["slot"] = _slots(g, n, n, s["pad"])
    s["table"] = torch.full_like(table, -1)
    s["table"][s["slot"][s["slot"] >= 0].long()] = table[s["slot"] >= 0]
    s["len"], s["counts"] = _ints(lens), _ints(counts)
    lead = (sum(counts),) if prompt else (n, T)
    # one projection's output row: q | k | v
    x = _randn(g, *lead, (H + 2 * kv) * d, dtype=s["dtype"])
    s["q"] = x[..., :H * d].unflatten(-1, (H, d))
    s["kx"] = x[..., H * d:(H + kv) * d].unflatten(-1, (kv, d))
    s["vx"] = x[..., (H + kv) * d:].unflatten(-1, (kv, d))
    s["wq"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(x.dtype)
    s["wk"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(x.dtype)
    s["cu"] = _cum(counts) if prompt else None
    at = torch.cat([torch.arange(c, device="cuda") for c in counts]) if prompt else \
        s["len"][:, None] + torch.arange(T, device="cuda")
    s["pos"] = (at + far).int().contiguous()
    s["k"] = torch.zeros(n_pages, page, kv, d, dtype=x.dtype, device="cuda")
    s["v"] = torch.zeros_like(s["k"])
    s["out"] = torch.zeros(*lead, H, d, dtype=x.dtype, device="cuda")
    _hold(s)
    return s


def _prepare_compact(s, g, seed):
    n, T, page = s["n_seq"], s["T"], s["page"]
    lens = _spread(n, 40, seed)
    table, n_pages = _table(g, [v + T for v in lens], page, extra=3)
    s["slot"] = _slots(g, n, n, s["pad"])
    s["table"] = torch.full_like(table, -1)
    s["table"][s["slot"][s["slot"] >= 0].long()] = table[s["slot"] >= 0]
    s["len"] = _ints(lens)
    s["k"] = _randn(g, s["layers"], n_pages, page, s["n_kv"], s["d"], dtype=s["dtype"])
    s["v"] = _randn(g, s["layers"], n_pages, page, s["n_kv"], s["d"], dtype=s["dtype"])
    # accepted paths: token 0 and a random choice of later ones, in order
    a = _ints(_spread(n, max(1, T // 2), seed, 1))
    key = torch.rand(n, T, generator=g, device="cuda")
    key[:, 0] = -1
    pick = key.argsort(1)
    i = torch.arange(T, device="cuda")
    s["path"] = torch.where(i < a[:, None], pick, T).sort(1).values.int()
    s["path"][i >= a[:, None]] = -1
    s["accept"] = a
    s["new_len"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    _hold(s)
    return s


def _prepare_fork(s, g, seed):
    """Sources in the first slots, then the continuations, which hold pages of an earlier fork."""
    n, m, page = s["n_dst"], s["n_src"], s["page"]
    lens = _spread(m, s["ctx"], seed, min(s["ctx"], 1))
    per = -(-(s["ctx"] + s["grow"]) // page)
    src = [i % m for i in range(n)]
    old = [max(1, -(-(lens[i] // 2) // page)) for i in src]
    shared = [min(o, lens[i] // page) for o, i in zip(old, src)]
    held = [-(-v // page) for v in lens]
    fresh = [o - c for o, c in zip(old, shared)]
    used = sum(held) + sum(fresh)
    n_pages = used + 2 * n * (2 + -(-s["grow"] // page))
    order = torch.randperm(n_pages, generator=g, device="cuda").cpu()
    table = torch.full((m + n, per), -1, dtype=torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        refs[order[at:at + h]] = 1
        at += h
    for j in range(n):
        table[m + j, :shared[j]] = table[src[j], :shared[j]]
        refs[table[src[j], :shared[j]].long()] += 1
        table[m + j, shared[j]:old[j]] = order[at:at + fresh[j]]
        refs[order[at:at + fresh[j]]] = 1
        at += fresh[j]
    s["table"], s["refs"] = table.cuda(), refs.cuda()
    s["held"] = _ints(held + old)
    s["src"], s["dst"] = _ints(src), _ints(list(range(m, m + n)))
    s["n_tok"] = _ints([lens[i] for i in src])
    s["grown"] = _ints([lens[i] + s["grow"] for i in src])
    s["k"] = _randn(g, s["layers"], n_pages, page, s["n_kv"], s["d"], dtype=s["dtype"])
    s["v"] = _randn(g, s["layers"], n_pages, page, s["n_kv"], s["d"], dtype=s["dtype"])
    _hold(s, held=s["held"], refs=s["refs"])
    return s


# ----------------------------------------------------------------------------------- plain forms


def _token_rows(table, pos, page):
    """Rows of the flattened cache at positions pos [n, L] of the sequences' table rows."""
    at = torch.gather(table.long(), 1, (pos // page).clamp(max=table.shape[1] - 1))
    return at.clamp(min=0) * page + pos % page


def _ancestors(parent, n, T):
    """[n, T, T]: whether token u is token t or an ancestor of it."""
    eye = torch.eye(T, dtype=torch.bool, device="cuda")
    if parent is None:
        return torch.ones(T, T, dtype=torch.bool, device="cuda").tril().expand(n, T, T)
    see = eye.expand(n, T, T).clone()
    for t in range(1, T):
        up = parent[:, t].long()
        above = see[torch.arange(n, device="cuda"), up.clamp(min=0)]
        see[:, t] |= above & (up >= 0)[:, None]
    return see


def _plain_attend(s):
    n, T, H, kv, d = s["n_seq"], s["T"], s["n_heads"], s["n_kv"], s["d"]
    live = s["slot"] >= 0
    L, counts = s["len"].long(), s["counts"].long()
    pos = torch.arange(s["top"], device="cuda").expand(n, -1)
    rows = _token_rows(s["table"][s["slot"].long().clamp(min=0)], pos, s["page"])
    ok = pos < (L + counts)[:, None]
    take = lambda c: torch.where(ok[..., None, None], c.flatten(0, 1)[rows], 0).transpose(1, 2).float()  # noqa: E731
    K, V = take(s["k"]), take(s["v"])
    t = torch.arange(T, device="cuda")
    if s["cu"] is not None:
        at = (s["cu"][:-1, None].long() + t).clamp(max=s["q"].shape[0] - 1)
        q = s["q"][at].float()
    else:
        q = s["q"].float()
    see = _ancestors(s["all_parents"], n, T)
    back = (pos - L[:, None])
    seen = torch.gather(see, 2, back.clamp(0, T - 1)[:, None, :].expand(n, T, s["top"]))
    seen = (seen & (back < counts[:, None])[:, None]) | (back < 0)[:, None]
    q = q.view(n, T, kv, H // kv, d).permute(0, 2, 1, 3, 4).reshape(n, kv, T * (H // kv), d)
    S = (q @ K.transpose(-1, -2)) * d ** -0.5
    S = S.masked_fill(~seen.repeat_interleave(H // kv, 1)[:, None], -math.inf)
    P = torch.exp(S - S.amax(-1, keepdim=True))
    P = P / P.sum(-1, keepdim=True)
    o = (P @ V).view(n, kv, T, H // kv, d).permute(0, 2, 1, 3, 4).reshape(n, T, H, d)
    if s["cu"] is not None:
        s["out"].copy_(o[t < counts[:, None]])
    else:
        s["out"].copy_(torch.where(live[:, None, None, None], o, 0.0))
    return s["out"]


def _plain_sample(s):
    n, T, V = s["n_seq"], s["T"], s["vocab"]
    seq, t = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    counts = s["counts"].long()[:, None]
    base = s["cu"][:-1, None].long() if s["cu"] is not None else seq[:, None] * T
    at = (base + t).clamp(max=s["tok"].numel() - 1)
    p, q = s["p"].view(-1, V), s["qp"].view(-1, V) if s["qp"] is not None else None
    tok = s["tok"].flatten()[at].long()
    up = s["all_parents"].long() if s["all_parents"] is not None else (t - 1).expand(n, T)
    up = torch.where(t < counts, up, -1)
    u = s["u"].double()
    mass = p[torch.gather(at, 1, up.clamp(min=0)), tok].double()
    path = torch.full((n, T), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    cur, a, going = torch.zeros_like(seq), torch.ones_like(seq), torch.ones_like(seq, dtype=torch.bool)
    twin = (tok[:, :, None] == tok[:, None, :]) & (up[:, :, None] == up[:, None, :])
    twin = (twin & torch.ones(T, T, dtype=torch.bool, device="cuda").tril(-1)).any(-1)
    for i in range(1, T):
        child = (up == cur[:, None]) & ~twin
        draw_ = u[seq, cur][:, None]
        if q is not None:
            ok = child & (draw_ * q[at, tok].double() < mass)
        else:
            ok = child & (draw_ < torch.where(child, mass, 0.0).cumsum(1))
        hit = ok.any(1) & going
        first = ok.int().argmax(1)
        path[:, i] = torch.where(hit, first, -1)
        cur, a, going = torch.where(hit, first, cur), a + hit, hit
    w = p[at[seq, cur]].double()
    own_ = w
    child = up == cur[:, None]
    if q is not None:
        row = torch.gather(at, 1, torch.where(child, t, 0).amax(1, keepdim=True))[:, 0]
        w = torch.where(child.any(1)[:, None], (w - q[row].double()).clamp(min=0), w)
    else:
        gone = torch.zeros(n, V + 1, dtype=torch.bool, device="cuda").scatter_(1, torch.where(child, tok, V), True)
        w = w.masked_fill(gone[:, :V], 0.0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, own_)
    c = w.cumsum(1)
    new = (c > u[:, T:] * c[:, -1:]).int().argmax(1)
    after = torch.cat([path[:, 1:], torch.full_like(path[:, :1], -1)], 1)
    out = torch.where(after >= 0, torch.gather(tok, 1, after.clamp(min=0)), -1)
    out[seq, a - 1] = new
    live = s["slot"] >= 0
    s["accept"].copy_(torch.where(live, a, 0))
    s["node"].copy_(torch.where(live, cur + 1, 0))
    s["new"].copy_(torch.where(live[:, None], out, 0))
    s["path"].copy_(torch.where(live[:, None], path, 0))
    return s["accept"], s["node"], s["new"], s["path"]


def _turned(x, w, cos, sin, pairs):
    """The norm over the last axis, then the rotation of its first 2 * cos.shape[-1] channels."""
    x = x.float()
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    half = cos.shape[-1]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (head[..., ::2], head[..., 1::2]) if pairs else (head[..., :half], head[..., half:])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([lo, hi], -1).flatten(-2) if pairs else torch.cat([lo, hi], -1)
    return torch.cat([head, rest], -1)


def _plain_rope(s):
    half = s["rot"] // 2
    cs = s["cos_sin"][s["pos"].long()].unsqueeze(-2)
    cos, sin = cs[..., :half], cs[..., half:]
    n, T = s["n_seq"], s["T"]
    if s["cu"] is not None:
        tok = torch.arange(s["q"].shape[0], device="cuda")
        seq = torch.searchsorted(s["cu"].long(), tok, right=True) - 1
        at = tok - s["cu"].long()[seq] + s["len"].long()[seq]
    else:
        seq = torch.arange(n, device="cuda").repeat_interleave(T)
        at = (s["len"][:, None] + torch.arange(T, device="cuda")).flatten()
    slot = s["slot"].long()[seq]
    live = slot >= 0
    q = _turned(s["q"], s["wq"], cos, sin, s["pairs"])
    keep = live.view(*s["q"].shape[:-2], 1, 1)
    s["out"].copy_(torch.where(keep, q, 0.0))
    rows = s["table"][slot.clamp(min=0), at // s["page"]].long() * s["page"] + at % s["page"]
    k = _turned(s["kx"], s["wk"], cos, sin, s["pairs"]).to(s["k"].dtype).flatten(0, -3)
    s["k"].flatten(0, 1)[rows[live]] = k[live]
    s["v"].flatten(0, 1)[rows[live]] = s["vx"].flatten(0, -3)[live]
    return s["out"], s["k"], s["v"]


def _plain_compact(s):
    n, T = s["n_seq"], s["T"]
    live = s["slot"] >= 0
    i = torch.arange(T, device="cuda")
    table = s["table"][s["slot"].long().clamp(min=0)]
    L = s["len"].long()[:, None]
    src = _token_rows(table, L + s["path"].long().clamp(min=0), s["page"])
    dst = _token_rows(table, L + i, s["page"])
    move = (i < s["accept"][:, None]) & live[:, None]
    src, dst = src[move], dst[move]
    for c in (s["k"], s["v"]):
        flat = c.flatten(1, 2)
        flat[:, dst] = flat[:, src]
    s["new_len"].copy_(torch.where(live, s["len"] + s["accept"], s["new_len"]))
    return s["k"], s["v"], s["new_len"]


def _take_pages(s, rows, first, count):
    """Table rows get count[i] of the lowest free pages at columns first[i]...; the pages' reference counts become 1."""
    free = (s["refs"] != 0).int().argsort(stable=True)
    before = count.cumsum(0) - count
    col = torch.arange(s["table"].shape[1], device="cuda")
    put = (col >= first[:, None]) & (col < (first + count)[:, None])
    pick = free[(before[:, None] + col - first[:, None])[put]]
    row = rows[:, None].expand_as(put)[put]
    s["table"][row, col.expand_as(put)[put]] = pick.int()
    s["refs"][pick] = 1


def _plain_fork(s):
    page, table, refs, held = s["page"], s["table"], s["refs"], s["held"]
    src, dst, n_tok = s["src"].long(), s["dst"].long(), s["n_tok"].long()
    col = torch.arange(table.shape[1], device="cuda")
    gone = col < held[dst][:, None]
    rows = table[dst]
    refs.index_add_(0, rows[gone].long(), -torch.ones_like(rows[gone]))
    table[dst] = torch.where(gone, -1, rows)
    held[dst] = 0
    full, rest = n_tok // page, n_tok % page
    _take_pages(s, dst, full, (rest > 0).long())
    shared = col < full[:, None]
    rows = table[src]
    refs.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    table[dst] = torch.where(shared, rows, table[dst])
    last = full.clamp(max=table.shape[1] - 1)
    copy = (torch.arange(page, device="cuda") < rest[:, None])
    old = (table[src, last].long().clamp(min=0) * page)[:, None] + torch.arange(page, device="cuda")
    new = (table[dst, last].long().clamp(min=0) * page)[:, None] + torch.arange(page, device="cuda")
    for c in (s["k"], s["v"]):
        flat = c.flatten(1, 2)
        flat[:, new[copy]] = flat[:, old[copy]]
    have = (n_tok + page - 1) // page
    want = (s["grown"].long() + page - 1) // page
    _take_pages(s, dst, have, want - have)
    held[dst] = want.int()
    return s["k"], s["v"], table, refs, held


def run(state):
    return _own(state) if own else _plain(state)


def _plain(s):
    return {"attend": _plain_attend, "sample": _plain_sample, "rope": _plain_rope, "compact": _plain_compact,
            "fork": _plain_fork}[s["op"]](s)


def _own(s):
    import spec_decode_verify_gb300 as cv
    if s["op"] == "attend":
        cv.tree_attention(s["q"], s["out"], s["cache"], s["len"], parent=s["parent"], cu_draft=s["cu"], T=s["T"],
                          cache_idx=s["slot"])
        return s["out"]
    if s["op"] == "sample":
        cv.draft_verify(s["p"], s["tok"], s["u"], s["accept"], s["new"], draft_probs=s["qp"], parent=s["parent"],
                        path=s["path"], accept_node=s["node"], cu_draft=s["cu"], T=s["T"], cache_idx=s["slot"])
        return s["accept"], s["node"], s["new"], s["path"]
    if s["op"] == "rope":
        cv.qk_norm_rope(s["q"], s["kx"], s["out"], cos_sin=s["cos_sin"], q_weight=s["wq"], k_weight=s["wk"], v=s["vx"],
                        cache=s["cache"], cache_len=s["len"], positions=s["pos"], cu_seqlens=s["cu"], max_seqlen=s["T"],
                        cache_idx=s["slot"], pairs=s["pairs"], eps=1e-6)
        return s["out"], s["k"], s["v"]
    if s["op"] == "compact":
        cv.cache_compact(s["cache"], s["len"], s["path"], s["accept"], new_len=s["new_len"], cache_idx=s["slot"])
        return s["k"], s["v"], s["new_len"]
    cv.cache_free(s["cache"], cache_idx=s["dst"])
    cv.cache_fork(s["cache"], s["src"], s["dst"], s["n_tok"])
    cv.cache_reserve(s["cache"], s["grown"], cache_idx=s["dst"])
    return s["k"], s["v"], s["table"], s["refs"], s["held"]


# ------------------------------------------------------------------------------------------ work


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "attend":
        counts, lens = _counts(case, 0), _spread(case["n_seq"], case["ctx"], 0)
        live = 1 - case["pad"] / case["n_seq"]
        keys = sum(v + c for v, c in zip(lens, counts)) * live
        new = sum(counts) * live
        seen = sum(c * v + c * (c + 1) / 2 for v, c in zip(lens, counts)) * live
        d, H, kv = case["d"], case["n_heads"], case["n_kv"]
        return {"bytes": keys * kv * d * 2 * e + new * H * d * 2 * e + keys / case["page"] * 4,
                "flops": 4 * seen * H * d}
    if op == "sample":
        live = case["n_seq"] - case["pad"]
        rows = 1.6 if case["q"] else 1  # a row of the target, and after a rejection (most walks end in one) the draft's
        return {"bytes": live * case["vocab"] * rows * e + live * case["T"] * 32, "flops": live * case["vocab"] * (1 + rows)}
    if op == "rope":
        tokens = sum(_counts(case, 0)) * (1 - case["pad"] / case["n_seq"])
        qk, kv = (case["n_heads"] + case["n_kv"]) * case["d"], case["n_kv"] * case["d"]
        return {"bytes": tokens * (2 * (qk + kv) * e + case["rot"] * 4 + 4), "flops": tokens * qk * 8}
    if op == "compact":
        moved = sum(v - 1 for v in _spread(case["n_seq"], max(1, case["T"] // 2), 0, 1)) * (1 - case["pad"] / case["n_seq"])
        return {"bytes": moved * case["layers"] * case["n_kv"] * case["d"] * 4 * e + case["n_seq"] * case["T"] * 8, "flops": 0}
    lens = _spread(case["n_src"], case["ctx"], 0, min(case["ctx"], 1))
    of = [lens[i % case["n_src"]] for i in range(case["n_dst"])]
    rest = sum(v % case["page"] for v in of)
    pages = sum(v // case["page"] + (v + case["grow"]) // case["page"] for v in of)
    return {"bytes": rest * case["layers"] * case["n_kv"] * case["d"] * 4 * e + pages * 24, "flops": 0}


# ----------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "sample": _exact_sample, "rope": _exact_rope, "compact": _exact_compact,
            "fork": _exact_fork}[case["op"]](s)


def _sequences(s):
    """(index, first row of the packed drafts, draft count, table row) of every sequence that is not padded."""
    slots, counts = s["slot"].tolist(), s["counts"].tolist()
    row = 0
    for i, (slot, c) in enumerate(zip(slots, counts)):
        if slot >= 0:
            yield i, (row if s["cu"] is not None else i * s["T"]), c, slot
        row += c


def _exact_attend(s):
    H, kv, d, page = s["n_heads"], s["n_kv"], s["d"], s["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    flat, q = out.view(-1, H, d), s["q"].reshape(-1, H, d)
    for i, row, c, slot in _sequences(s):
        L = int(s["len"][i])
        pages = s["table"][slot, :-(-(L + c) // page)].long()
        K = s["k"][pages].flatten(0, 1)[:L + c].double()
        V = s["v"][pages].flatten(0, 1)[:L + c].double()
        up = s["all_parents"][i].tolist() if s["all_parents"] is not None else list(range(-1, c - 1))
        for t in range(c):
            seen = []
            at = t
            while at >= 0:
                seen.append(L + at)
                at = up[at]
            seen = torch.tensor(list(reversed(seen)), device="cuda")
            for h in range(kv):
                x = q[row + t, h * H // kv:(h + 1) * H // kv].double()
                w = torch.softmax(torch.cat([x @ K[:L, h].T, x @ K[seen, h].T], 1) / math.sqrt(d), 1)
                flat[row + t, h * H // kv:(h + 1) * H // kv] = w[:, :L] @ V[:L, h] + w[:, L:] @ V[seen, h]
    return out


def _exact_sample(s):
    n, T, V = s["n_seq"], s["T"], s["vocab"]
    accept, node = [0] * n, [0] * n
    new, path = [[0] * T for _ in range(n)], [[0] * T for _ in range(n)]
    toks, u = s["tok"].flatten().tolist(), s["u"].double().tolist()
    p, q = s["p"].view(-1, V), s["qp"].view(-1, V) if s["qp"] is not None else None
    for i, row, c, _ in _sequences(s):
        up = s["all_parents"][i].tolist() if s["all_parents"] is not None else list(range(-1, c - 1))
        walk = [0]
        while True:
            cur = walk[-1]
            kids = [t for t in range(c) if up[t] == cur]
            target = p[row + cur].double()
            took, sofar, tried = None, 0.0, set()
            for t in kids:
                x = toks[row + t]
                if x in tried:
                    continue
                tried.add(x)
                if q is not None:
                    good = u[i][cur] * float(q[row + t, x]) < float(target[x])
                else:
                    sofar += float(target[x])
                    good = u[i][cur] < sofar
                if good:
                    took = t
                    break
            if took is None:
                break
            walk.append(took)
        w = target.clone()
        if kids and q is not None:
            w = (target - q[row + kids[-1]].double()).clamp(min=0)
        elif kids:
            w[[toks[row + t] for t in kids]] = 0
        if float(w.sum()) <= 0:
            w = target
        sums = torch.cumsum(w, 0)
        token = int(torch.searchsorted(sums, (u[i][T] * sums[-1]).view(1), right=True))
        accept[i], node[i] = len(walk), walk[-1] + 1
        path[i] = walk + [-1] * (T - len(walk))
        new[i] = [toks[row + t] for t in walk[1:]] + [token] + [-1] * (T - len(walk))
    return _ints(accept), _ints(node), _ints(new), _ints(path)


def _exact_rope(s):
    half, d = s["rot"] // 2, s["d"]

    def turned(x, w, pos):
        x = x.double()
        x = x * (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).pow(-0.5) * w.double()
        z = s["cos_sin"][pos.long()].double()
        z = torch.complex(z[:, :half], z[:, half:]).unsqueeze(1)
        y = x.clone()
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["pairs"] else (slice(0, half), slice(half, 2 * half))
        c = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = c.real, c.imag
        return y

    out, K, V = s["out"].double(), s["k"].double(), s["v"].double()
    flat = [t.reshape(-1, *t.shape[-2:]) for t in (s["q"], s["kx"], s["vx"])]
    pos = s["pos"].flatten()
    for i, row, c, slot in _sequences(s):
        sl = slice(row, row + c)
        out.view(-1, *out.shape[-2:])[sl] = turned(flat[0][sl], s["wq"], pos[sl])
        at = int(s["len"][i]) + torch.arange(c, device="cuda")
        page, col = s["table"][slot].long()[at // s["page"]], at % s["page"]
        K[page, col] = turned(flat[1][sl], s["wk"], pos[sl])
        V[page, col] = flat[2][sl].double()
    return out, K, V


def _exact_compact(s):
    k, v, new_len, page = s["k"].clone(), s["v"].clone(), s["new_len"].clone(), s["page"]
    path, accept, lens, table = s["path"].tolist(), s["accept"].tolist(), s["len"].tolist(), s["table"].tolist()
    src, dst = [], []
    for i, slot in enumerate(s["slot"].tolist()):
        if slot < 0:
            continue
        new_len[i] = lens[i] + accept[i]
        for j in range(accept[i]):
            for to, at in ((src, lens[i] + path[i][j]), (dst, lens[i] + j)):
                to.append((table[slot][at // page], at % page))
    (a, b), (c, d) = (torch.tensor(x, device="cuda").T for x in (src, dst))
    k[:, c, d], v[:, c, d] = s["k"][:, a, b], s["v"][:, a, b]
    return k, v, new_len


def _exact_fork(s):
    page = s["page"]
    table, refs, held = s["table"].tolist(), s["refs"].tolist(), s["held"].tolist()
    k, v = s["k"].clone(), s["v"].clone()
    src, dst, n_tok, grown = (s[x].tolist() for x in ("src", "dst", "n_tok", "grown"))
    for d in dst:
        for c in range(held[d]):
            refs[table[d][c]] -= 1
            table[d][c] = -1
        held[d] = 0
    for a, d, n in zip(src, dst, n_tok):
        if n % page:
            f = refs.index(0)
            refs[f], table[d][n // page] = 1, f
    for a, d, n in zip(src, dst, n_tok):
        for c in range(n // page):
            table[d][c] = table[a][c]
            refs[table[a][c]] += 1
        if n % page:
            to, frm = table[d][n // page], table[a][n // page]
            k[:, to, :n % page], v[:, to, :n % page] = s["k"][:, frm, :n % page], s["v"][:, frm, :n % page]
        held[d] = -(-n // page)
    for d, n in zip(dst, grown):
        for c in range(held[d], -(-n // page)):
            f = refs.index(0)
            refs[f], table[d][c] = 1, f
        held[d] = max(held[d], -(-n // page))
    return k, v, _ints(table), _ints(refs), _ints(held)
