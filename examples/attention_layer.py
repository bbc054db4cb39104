"""One attention layer of a hybrid model served with speculative decoding: a paged cache, drafted trees, and their acceptance.

    python examples/attention_layer.py

    prompt   cache_reserve -> qk_norm_rope (K and V into the cache's pages) -> tree_attention, in chunks of drafts without parents
    step     the same over a tree of T drafts, each attending to the cached tokens and its ancestors; draft_verify says from the
             target's probabilities which of them stand; cache_compact moves their K and V to their places, and cache_free gives the tail's pages
             back.  cache_fork lets a second sequence go on from the first one's tokens.

Weights, tokens and probabilities are random.  At the end the accepted tokens are run once more as one long prompt: the cache holds the
same bits, and the outputs agree within bf16.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spec_decode_verify_gb300 as cv  # noqa: E402

CHUNK = 128  # tokens a call of tree_attention takes for a sequence


class AttentionLayer:
    def __init__(self, n_heads=16, n_kv=4, d=128, page=16, slots=4, max_pages=32, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.n_heads, self.n_kv, self.d = n_heads, n_kv, d
        shape = (slots * max_pages, page, n_kv, d)
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
        self.cache = cv.PagedCache(torch.zeros(shape, dtype=torch.bfloat16, device=device), torch.zeros(shape, dtype=torch.bfloat16, device=device),
                                   ints(slots, max_pages) - 1, held=ints(slots), refs=ints(slots * max_pages))
        self.len = ints(slots)
        self.wq, self.wk = ((1 + 0.1 * torch.randn(d, generator=g, device=device)).bfloat16() for _ in range(2))
        angle = torch.arange(max_pages * page, device=device, dtype=torch.float64)[:, None] * \
            1e6 ** (-torch.arange(d // 2, device=device, dtype=torch.float64) * 2 / d)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()

    def run(self, x, slots, parent=None, depth=None):
        """x [n_seq, T, (n_heads + 2 n_kv) d]: one projection's rows.  The drafts' K and V go behind the cached tokens."""
        n, T = x.shape[:2]
        H, kv, d = self.n_heads, self.n_kv, self.d
        lens = self.len[slots.long()]
        cv.cache_reserve(self.cache, lens + T, cache_len=lens, cache_idx=slots)
        q = x[..., :H * d].unflatten(-1, (H, d))
        k, v = (x[..., (H + i * kv) * d:(H + (i + 1) * kv) * d].unflatten(-1, (kv, d)) for i in range(2))
        turned, out = torch.empty(n, T, H, d, dtype=x.dtype, device=x.device), torch.empty(n, T, H, d, dtype=x.dtype, device=x.device)
        # a draft's position is its depth in the tree; its place in the cache is its number
        at = (lens[:, None] + depth).int() if depth is not None else None
        cv.qk_norm_rope(q, k, turned, v=v, cos_sin=self.cos_sin, q_weight=self.wq, k_weight=self.wk, positions=at, cache=self.cache,
                        cache_len=lens, cache_idx=slots)
        cv.tree_attention(turned, out, self.cache, lens, parent=parent, cache_idx=slots)
        return out

    def prompt(self, x, slots):
        """x [n_seq, length, ...], a chunk at a time."""
        outs = []
        for t in range(0, x.shape[1], CHUNK):
            part = x[:, t:t + CHUNK]
            outs.append(self.run(part, slots))
            self.len[slots.long()] += part.shape[1]
        return torch.cat(outs, 1)

    def accept(self, slots, path, accepted):
        """The accepted path's K and V to their places; what is behind them goes."""
        lens = self.len[slots.long()]
        new = torch.empty_like(lens)
        cv.cache_compact(self.cache, lens, path, accepted, new_len=new, cache_idx=slots)
        cv.cache_free(self.cache, new, cache_idx=slots)
        self.len[slots.long()] = new

    def rows(self, slot):
        """K and V of a slot's tokens."""
        n, page = int(self.len[slot]), self.cache.k.shape[1]
        at = torch.arange(n, device=self.len.device)
        pages = self.cache.page_table[slot].long()[at // page]
        return self.cache.k[pages, at % page], self.cache.v[pages, at % page]


def main(n_seq=2, prompt=150, T=8, steps=4, vocab=1000, seed=0):
    """Serves prompts, a fork and a few steps.  Returns the outputs' largest difference to one long prompt, the largest size of an
    output, a key or a value, and the largest difference of the cached keys and values."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    layer, check = AttentionLayer(seed=seed), AttentionLayer(seed=seed)
    width = (layer.n_heads + 2 * layer.n_kv) * layer.d
    slots = torch.tensor([2, 0], dtype=torch.int32, device=dev)[:n_seq]
    x = torch.randn(n_seq, prompt, width, generator=g, device=dev).bfloat16()
    outs = layer.prompt(x, slots)
    # a third sequence goes on from the first one's prompt
    fork = torch.tensor([3], dtype=torch.int32, device=dev)
    cv.cache_fork(layer.cache, slots[:1].clone(), fork, layer.len[slots[:1].long()])
    layer.len[3] = layer.len[int(slots[0])]
    slots = torch.cat([slots, fork])
    kept_x = [[x[s]] for s in range(n_seq)] + [[x[0]]]
    kept_out = [[outs[s]] for s in range(n_seq)] + [[outs[0]]]
    n = n_seq + 1

    parent = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 6][:T]] * n, dtype=torch.int32, device=dev)
    depth = torch.zeros(T, dtype=torch.int32, device=dev)
    for t in range(1, T):
        depth[t] = depth[parent[0, t]] + 1
    for _ in range(steps):
        x = torch.randn(n, T, width, generator=g, device=dev).bfloat16()
        out = layer.run(x, slots, parent, depth)
        probs = torch.softmax(2 * torch.randn(n, T, vocab, generator=g, device=dev), -1)
        up = parent.long().clamp(min=0)
        tokens = torch.multinomial(probs[torch.arange(n, device=dev)[:, None], up].view(-1, vocab).pow(2), 1, generator=g).view(n, T).int()
        accepted, path, new = (torch.empty(*s, dtype=torch.int32, device=dev) for s in ((n,), (n, T), (n, T)))
        cv.draft_verify(probs, tokens, torch.rand(n, T + 1, generator=g, device=dev) * 0.05, accepted, new, parent=parent, path=path)
        layer.accept(slots, path, accepted)
        for s in range(n):
            at = path[s, :int(accepted[s])].long()
            kept_x[s].append(x[s, at])
            kept_out[s].append(out[s, at])

    d_out = top = d_cache = 0.0
    for s in range(n):  # the same tokens as one prompt
        rows = torch.cat(kept_x[s])[None]
        want = check.prompt(rows, torch.tensor([s], dtype=torch.int32, device=dev))[0].float()
        d_out = max(d_out, float((torch.cat(kept_out[s]).float() - want).abs().max()))
        top = max(top, float(want.abs().max()))
        for a, b in zip(layer.rows(int(slots[s])), check.rows(s)):
            top = max(top, float(b.float().abs().max()))
            d_cache = max(d_cache, float((a.float() - b.float()).abs().max()))
    return d_out, top, d_cache


if __name__ == "__main__":
    d_out, top, d_cache = main()
    print(f"drafted trees accepted step by step against one long prompt: outputs differ by at most {d_out:.3g} "
          f"(values up to {top:.3g}), "
          f"cached keys and values by {d_cache:.2g}")
