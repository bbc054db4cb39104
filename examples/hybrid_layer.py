"""One hybrid layer served with speculative decoding: every operator of the library where a program calls it.

    python examples/hybrid_layer.py

A layer holds conv weights over q|k|v channels, linear attention with a decay for each head, a gated norm for
each head, an output projection, and the norms around the block; the residual stream is fp32.

    prompt   conv_prefill -> linattn_prefill -> block_norm (per-head, gated) -> projection
             -> block_norm (post-norm, scaled residual, the next block's pre-norm)
    step     the same over T draft tokens with conv_verify and linattn_step; the tokens the model accepts are
             committed by conv_commit, and by the next linattn_step before it reads the state

Weights and tokens are random.  At the end the accepted tokens are run once more as one long prompt: outputs
and states agree within bf16, however the drafts were accepted.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spec_decode_verify_gb300 as cv  # noqa: E402


class HybridLayer:
    def __init__(self, hidden=1024, n_qk=4, n_heads=8, dk=128, dv=128, width=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.n_qk, self.n_heads, self.dk, self.dv, self.width = hidden, n_qk, n_heads, dk, dv, width
        self.qk, self.v = 2 * n_qk * dk, n_heads * dv

        def w(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).bfloat16()

        self.w_in = w(hidden, self.qk + 2 * self.v + n_heads, scale=hidden ** -0.5)  # q|k|v, gate, decay
        self.w_conv = w(self.qk + self.v, width, scale=0.5)
        self.w_out = w(self.v, hidden, scale=self.v ** -0.5)
        self.norm_head = 1 + w(dv, scale=0.1)
        self.norm_post, self.norm_next = 1 + w(hidden, scale=0.1), 1 + w(hidden, scale=0.1)

    def states(self, n_slots):
        """Conv windows and attention states of n_slots sequences."""
        dev = self.w_in.device
        return (torch.zeros(n_slots, self.qk + self.v, self.width - 1, dtype=torch.bfloat16, device=dev),
                torch.zeros(n_slots, self.n_heads, self.dk, self.dv, device=dev))

    def project(self, x):
        """x [.., hidden] -> conv input, gate [.., v], log decay fp32 [.., heads]."""
        y = x @ self.w_in
        conv, gate, a = y.split([self.qk + self.v, self.v, self.n_heads], -1)
        return conv, gate, -torch.nn.functional.softplus(a.float() - 3.0)

    def heads(self, y):
        """q, k, v views of the conv's output rows."""
        k0 = self.qk // 2
        return (y[..., :k0].unflatten(-1, (self.n_qk, self.dk)), y[..., k0:self.qk].unflatten(-1, (self.n_qk, self.dk)),
                y[..., self.qk:].unflatten(-1, (self.n_heads, self.dv)))

    def finish(self, attn, gate, residual):
        """Gated norm of each head, projection, and the norms around the block.  Returns the next block's input and
        the new residual stream."""
        rows = attn.reshape(-1, self.v)
        cv.block_norm(rows, rows, gate=gate.reshape(-1, self.v), group=self.dv, post_weight=self.norm_head)
        y = rows @ self.w_out
        res = residual.reshape(-1, self.hidden)
        new, nxt = torch.empty_like(res), torch.empty_like(y)
        cv.block_norm(y, nxt, group=self.hidden, post_weight=self.norm_post, residual=res, residual_out=new, scale=0.5,
                      pre_weight=self.norm_next)
        return nxt.view(*residual.shape), new.view(residual.shape)

    def prompt(self, x, residual, cu, max_len, conv_state, state, slots):
        """Packed prompts x [total, hidden] from empty states."""
        conv_in, gate, g = self.project(x)
        conv = torch.empty_like(conv_in, memory_format=torch.contiguous_format)
        fresh = torch.zeros(len(slots), dtype=torch.int32, device=x.device)
        cv.conv_prefill(conv_in, conv_state, self.w_conv, None, conv, cu, max_seqlen=max_len, qk_channels=self.qk,
                        head_dim=self.dk, cache_idx=slots, has_initial_state=fresh)
        q, k, v = self.heads(conv)
        attn = torch.empty(x.shape[0], self.n_heads, self.dv, dtype=x.dtype, device=x.device)
        cv.linattn_prefill(q, k, v, g, state, attn, cu, max_seqlen=max_len, cache_idx=slots, has_initial_state=fresh)
        return self.finish(attn, gate, residual)

    def verify(self, x, residual, conv_state, state, slots, prev=None):
        """T draft tokens a sequence, x [n_seq, T, hidden]; prev: the last step's drafts, committed on the way.
        Returns the outputs, the conv's input (its commit rebuilds the window from it), and the drafts."""
        conv_in, gate, g = self.project(x)
        conv_in = conv_in.contiguous()
        conv = torch.empty_like(conv_in)
        cv.conv_verify(conv_in, conv_state, self.w_conv, None, conv, None, layout="recompute", qk_channels=self.qk,
                       head_dim=self.dk, cache_idx=slots)
        q, k, v = self.heads(conv)
        attn = torch.empty(*x.shape[:2], self.n_heads, self.dv, dtype=x.dtype, device=x.device)
        cv.linattn_step(q, k, v, g, state, attn, update_state=False, prev=prev, cache_idx=slots)
        nxt, res = self.finish(attn, gate, residual)
        return nxt, res, conv_in, (k, v, g)

    def accept(self, conv_in, drafts, accept_len, conv_state, slots):
        """The accepted prefix: the conv's window now, the attention state with the next step."""
        cv.conv_commit(conv_state, None, accept_len, layout="recompute", T=conv_in.shape[1], width=self.width, x=conv_in,
                       cache_idx=slots)
        return cv.LinattnDrafts(*drafts, accept_len)


def main(n_seq=3, prompt=(37, 200, 150), T=4, steps=3, seed=0):
    """Serves prompts and a few verify steps; returns the largest differences to one long prompt."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    layer = HybridLayer(seed=seed)
    conv_state, state = layer.states(n_seq + 1)
    slots = torch.tensor(list(range(n_seq, 0, -1)), dtype=torch.int32, device=dev)
    cu = torch.tensor([0] + list(prompt), device=dev).cumsum(0).int()
    x = torch.randn(sum(prompt), layer.hidden, generator=g, device=dev).bfloat16()
    out, _ = layer.prompt(x, x.float(), cu, max(prompt), conv_state, state, slots)
    lo = cu.tolist()
    kept_in = [[x[lo[s]:lo[s + 1]]] for s in range(n_seq)]
    kept_out = [[out[lo[s]:lo[s + 1]]] for s in range(n_seq)]

    prev = None
    for _ in range(steps):
        x = torch.randn(n_seq, T, layer.hidden, generator=g, device=dev).bfloat16()
        out, _, conv_in, drafts = layer.verify(x, x.float(), conv_state, state, slots, prev)
        accepted = torch.randint(1, T + 1, (n_seq,), generator=g, device=dev).int()
        prev = layer.accept(conv_in, drafts, accepted, conv_state, slots)
        for s, a in enumerate(accepted.tolist()):
            kept_in[s].append(x[s, :a])
            kept_out[s].append(out[s, :a])
    cv.linattn_commit(prev, state, cache_idx=slots)

    # the same tokens as prompts
    rows = [torch.cat(r) for r in kept_in]
    cu = torch.tensor([0] + [len(r) for r in rows], device=dev).cumsum(0).int()
    conv2, state2 = layer.states(n_seq + 1)
    x = torch.cat(rows)
    want, _ = layer.prompt(x, x.float(), cu, max(len(r) for r in rows), conv2, state2, slots)
    got = torch.cat([torch.cat(r) for r in kept_out])
    d_out = float((got.float() - want.float()).abs().max())
    d_state = float((state - state2).abs().max() / state2.abs().max())
    d_conv = float((conv_state.float() - conv2.float()).abs().max())
    return d_out, d_state, d_conv


if __name__ == "__main__":
    d_out, d_state, d_conv = main()
    print(f"drafts accepted step by step against one long prompt: outputs differ by at most {d_out:.3g}, "
          f"attention states by {d_state:.2g} of their largest value, conv windows by {d_conv:.2g}")
