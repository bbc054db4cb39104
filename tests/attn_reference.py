"""Plain 64-bit forms of the attention layers' operators, sequence by sequence on the CPU, for the tests."""
from __future__ import annotations

import math

import torch


def ancestors(parent):
    """Of each draft: itself and its ancestors, in order."""
    seen = []
    for t, p in enumerate(parent):
        seen.append((seen[p] if p >= 0 else []) + [t])
    return seen


def chain(T):
    return list(range(-1, T - 1))


def gather(cache, table_row, n):
    """Rows 0..n-1 of a sequence: [n, n_kv, d] in fp64."""
    page = cache.shape[1]
    at = torch.arange(n)
    return cache[table_row[at // page].long(), at % page].double()


def attention(q, K, V, L, parent, scale):
    """q [T, H, d], K and V [L + T, n_kv, d] in fp64.  Returns out, the mean of |v| with the same weights, and the largest
    scale * sum |q| |k| of each row: what the bounds of an error are made of."""
    T, H, d = q.shape
    kv = K.shape[1]
    out, size, top = torch.zeros(T, H, d, dtype=torch.float64), torch.zeros(T, H, d, dtype=torch.float64), torch.zeros(T, H, 1, dtype=torch.float64)
    for t, seen in enumerate(ancestors(parent)):
        keys = list(range(L)) + [L + u for u in seen]
        for h in range(H):
            k, v, x = K[keys, h * kv // H], V[keys, h * kv // H], q[t, h].double()
            w = torch.softmax(scale * (k @ x), 0)
            out[t, h] = (w[:, None] * v).sum(0)
            size[t, h] = (w[:, None] * v.abs()).sum(0)
            top[t, h] = scale * (k.abs() @ x.abs()).max()
    return out, size, top


def attention_bound(dtype, out, size, top, keys, d):
    """A bound on the error of fp32 arithmetic with one rounding of the result, and for bf16 one of each weight.

    A score is a sum of d products, scaled: each of its d + 2 fp32 operations is off by at most 2^-23 of top (twice half a
    step, for sums that are cut off), and so is what the weight's exponent is made of, at most top * log2(e) in size; exp2 is
    within 2^-22 of itself.  So a weight is off by e = (d + 6) 2^-23 top + 2^-22 of itself, and the sum over `keys` of them in
    fp32, with its rescaling, by (keys + 8) 2^-23 more.  Numerator and denominator both: twice.  The weights' rounding to
    bf16 adds 2^-8 of the numerator, the result's 2^-8 or 2^-24 of itself."""
    e = (d + 6) * 2.0 ** -23 * top + 2.0 ** -22 + (keys + 8) * 2.0 ** -23
    if dtype == torch.bfloat16:
        return 2.0 ** -8 * out.abs() + size * (2.0 ** -8 + 2 * e) * (1 + 2.0 ** -7)
    return 2.0 ** -24 * out.abs() + size * 2 * e * 1.01


def verify(p, tokens, uniforms, parent, q=None):
    """p [T, vocab], tokens, uniforms [T + 1] (the last one samples).  Returns the path and the new token."""
    T = len(tokens)
    path = [0]
    while True:
        c = path[-1]
        kids, tried, went, total = [t for t in range(T) if parent[t] == c], [], None, 0.0
        last = None
        for t in kids:
            x = tokens[t]
            if x in tried:
                continue
            last = t
            mass = float(p[c, x])
            total += mass
            if (float(uniforms[c]) * float(q[t, x]) < mass) if q is not None else (float(uniforms[c]) < total):
                went = t
                break
            tried.append(x)
        if went is None:
            break
        path.append(went)
    row = p[c].double().clamp(min=0)
    w = row.clone()
    if kids and q is not None:
        w = (row - q[last].double().clamp(min=0)).clamp(min=0)
    elif kids:
        w[tried] = 0
    if float(w.sum()) == 0:
        w = row
    sums = w.cumsum(0)
    return path, int(torch.nonzero(sums > float(uniforms[-1]) * sums[-1])[0])


def norm_rope(x, weight, cos, sin, pairs, norm, eps):
    """x [.., heads, d], cos and sin [.., rot / 2], in fp64."""
    x = x.double()
    if norm:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    half = cos.shape[-1]
    cos, sin = cos.double().unsqueeze(-2), sin.double().unsqueeze(-2)
    y = x.clone()
    a = torch.arange(half) * 2 if pairs else torch.arange(half)
    b = a + 1 if pairs else a + half
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


class Pool:
    """The pages' bookkeeping, one call after the other, on lists."""

    def __init__(self, table, held, refs, page):
        self.table, self.held, self.refs, self.page = [list(r) for r in table], list(held), list(refs), page

    def pages(self, n):
        return -(-n // self.page)

    def take(self):
        f = self.refs.index(0)
        self.refs[f] = 1
        return f

    def reserve(self, idx, n_tokens):
        err, named, room, out = [], set(), self.refs.count(0), False
        for slot, n in zip(idx, n_tokens):
            e = 0
            if slot >= 0:
                need = max(0, self.pages(n) - self.held[slot]) if 0 <= slot < len(self.table) else 0
                if slot >= len(self.table) or slot in named:
                    e, need = 1, 0
                elif n < 0 or n > len(self.table[0]) * self.page:
                    e, need = 64, 0
                named.add(slot)
                if need:
                    out = out or need > room
                    if out:
                        e = 1024
                    else:
                        room -= need
                        for c in range(need):
                            self.table[slot][self.held[slot] + c] = self.take()
                        self.held[slot] += need
            err.append(e)
        return err

    def fork(self, src, dst, n_tokens):
        """Returns err and the (new page, old page, rows) to copy."""
        err, copies, todo, named = [], [], [], set()
        sources = {a for a, d in zip(src, dst) if a >= 0 and d >= 0}
        room, held = self.refs.count(0), list(self.held)
        for a, d, n in zip(src, dst, n_tokens):
            e = 0
            if a >= 0 and d >= 0:
                if d >= len(self.table) or a >= len(self.table) or d in named or d in sources or held[d]:
                    e = 1
                elif n < 0 or n > held[a] * self.page:
                    e = 64
                elif n % self.page and not room:
                    e = 1024
                named.add(d)
                if not e:
                    room -= n % self.page != 0
                    todo.append((a, d, n, self.take() if n % self.page else None))
            err.append(e)
        for a, d, n, f in todo:
            full = n // self.page
            for c in range(full):
                self.table[d][c] = self.table[a][c]
                self.refs[self.table[a][c]] += 1
            if f is not None:
                self.table[d][full] = f
                copies.append((f, self.table[a][full], n % self.page))
            self.held[d] = self.pages(n)
        return err, copies

    def free(self, idx, n_tokens):
        err, named = [], set()
        for slot, n in zip(idx, n_tokens):
            e = 0
            if slot >= 0:
                if slot >= len(self.table) or slot in named:
                    e = 1
                elif n < 0:
                    e = 64
                else:
                    for c in range(self.pages(n), self.held[slot]):
                        self.refs[self.table[slot][c]] -= 1
                        self.table[slot][c] = -1
                    self.held[slot] = min(self.held[slot], self.pages(n))
                named.add(slot)
            err.append(e)
        return err


def decaying(n, vocab, g, sharp=3.0):
    """n distributions of a few likely values and a tail, fp32."""
    return torch.softmax(torch.randn(n, vocab, generator=g) * sharp, -1)


assert math.isclose(2.0 ** -8, torch.finfo(torch.bfloat16).eps / 2)
