"""A transformer block's attention half on the library: training step, prefill and decoding.

    python examples/attention_block.py            # on an MI355X

Per token the projection gives a row [Q | K | V]; the short convolution runs on
it with filters generated from the hidden state, fused with the rotary
embedding of Q and K; causal attention with grouped heads follows.  The same
weights then serve: packed prompts fill a paged key-value cache, and each new
token takes one convolution step, one append and one attention over the cache.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from input_dependent_short_amd import binding as dsc  # noqa: E402


class AttentionBlock:
    """Weights of one block: projection, filter generator, output projection (bf16, on the GPU)."""

    def __init__(self, width=512, q_heads=8, kv_heads=2, head_dim=64, taps=4, group=16, max_pos=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.hd, self.W, self.H = q_heads, kv_heads, head_dim, taps, group
        self.D = (q_heads + 2 * kv_heads) * head_dim
        self.rot = (q_heads + kv_heads) * head_dim  # channels the rotary embedding turns
        new = lambda n, k, s: (torch.randn(n, k, generator=g, device="cuda") * s).bfloat16()
        self.w_qkv = new(self.D, width, width ** -0.5)
        self.w_gen = new(self.D // group * taps, width, (width * taps) ** -0.5)
        self.w_out = new(width, q_heads * head_dim, (q_heads * head_dim) ** -0.5)
        self.table = torch.empty(max_pos, head_dim // 2, 2, device="cuda")
        dsc.dsc_rope_table(self.table)

    def heads(self, row):
        """q, k, v views of [Q | K | V] rows."""
        q, k, v = row.split([self.Hq * self.hd, self.Hkv * self.hd, self.Hkv * self.hd], dim=-1)
        return (t.unflatten(-1, (-1, self.hd)) for t in (q, k, v))

    def rows(self, x):
        """Projection rows and their filters (B, T, D/H, W) of the hidden states x (B, T, width)."""
        w = torch.empty(*x.shape[:2], self.D // self.H, self.W, dtype=x.dtype, device=x.device)
        dsc.dsc_generate_filters(x, self.w_gen, w)
        return x @ self.w_qkv.T, w

    def forward(self, x, cu=None):
        """Output (B, T, width) and what the backward and the cache need."""
        row, w = self.rows(x)
        y = torch.empty_like(row)
        dsc.dsc_headwise_rope_fwd(row, w, y, rot=self.rot, head_dim=self.hd, table=self.table, cu_seqlens=cu, residual=True)
        q, k, v = self.heads(y)
        B, T = x.shape[:2]
        o = torch.empty(B, T, self.Hq, self.hd, dtype=x.dtype, device=x.device)
        lse = torch.empty(self.Hq, B * T, device=x.device)
        dsc.dsc_attn_fwd(q, k, v, o, lse, cu_seqlens=cu)
        return o.flatten(-2) @ self.w_out.T, (row, w, y, o, lse)

    def backward(self, x, kept, dout, cu=None):
        """Gradients of the three weights for dL/d(output) = dout."""
        row, w, y, o, lse = kept
        B, T = x.shape[:2]
        do = (dout @ self.w_out).unflatten(-1, (self.Hq, self.hd)).contiguous()
        dy = torch.empty_like(y)
        n = dsc.dsc_attn_bwd_workspace_size(x.dtype, B, T, self.Hq, self.Hkv, self.hd)
        dsc.dsc_attn_bwd(*self.heads(y), o, lse, do, *self.heads(dy), torch.empty(n, dtype=torch.uint8, device="cuda"),
                         cu_seqlens=cu)
        drow, dw = torch.empty_like(row), torch.empty_like(w)
        dsc.dsc_headwise_rope_bwd(row, w, dy, drow, dw, rot=self.rot, head_dim=self.hd, table=self.table, cu_seqlens=cu,
                                  residual=True)
        flat = lambda t: t.reshape(B * T, -1).float()
        return {"w_qkv": flat(drow).T @ flat(x), "w_gen": flat(dw).T @ flat(x), "w_out": flat(dout).T @ flat(o)}


class Cache:
    """A paged key-value cache and the convolution's state of a batch of sequences."""

    def __init__(self, block, sequences, max_len, page=64):
        b, per = block, -(-max_len // page)
        self.k = torch.empty(sequences * per, b.Hkv, page, b.hd, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        self.pages = torch.randperm(sequences * per, device="cuda").to(torch.int32).view(sequences, per)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.state = torch.zeros(sequences, b.W - 1, b.D, dtype=torch.bfloat16, device="cuda")
        n = dsc.dsc_attn_decode_workspace_size(torch.bfloat16, sequences, b.Hq, b.Hkv, b.hd, page, per)
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def prefill(self, block, x, cu):
        """Packed prompts x (1, N, width) with offsets cu: outputs, and the cache filled."""
        out, (row, _, y, _, _) = block.forward(x, cu)
        _, k, v = block.heads(y[0])
        dsc.dsc_kv_append(k, v, self.k, self.v, self.pages, self.lens, cu_seqlens=cu)  # rotated already
        dsc.dsc_state_from_prefill(row, self.state, W=block.W, cu_seqlens=cu)
        self.lens += cu[1:] - cu[:-1]
        return out

    def step(self, block, x):
        """One new token per sequence, x (S, width): its output (S, width)."""
        row, w = block.rows(x[:, None])
        y = torch.empty_like(row[:, 0])
        dsc.dsc_headwise_rope_decode(row[:, 0].contiguous(), w[:, 0].contiguous(), self.state, y, self.lens, rot=block.rot,
                                     head_dim=block.hd, table=block.table, residual=True)
        q, k, v = block.heads(y)
        dsc.dsc_kv_append(k, v, self.k, self.v, self.pages, self.lens)
        self.lens += 1
        o = torch.empty(x.shape[0], block.Hq, block.hd, dtype=x.dtype, device=x.device)
        dsc.dsc_attn_decode(q, self.k, self.v, self.pages, self.lens, o, self.ws)
        return o.flatten(-2) @ block.w_out.T


def train(block, steps=30, B=2, T=384, lr=2e-3, seed=1):
    """Fits a random target by sign descent on the block's weights; the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, T, block.w_qkv.shape[1], generator=g, device="cuda").bfloat16()
    want = torch.randn(x.shape, generator=g, device="cuda").bfloat16() * 0.5
    losses = []
    for _ in range(steps):
        out, kept = block.forward(x)
        diff = out.float() - want.float()
        losses.append(float(diff.square().mean()))
        for name, grad in block.backward(x, kept, (2.0 * diff / diff.numel()).bfloat16()).items():
            w = getattr(block, name)
            w.copy_((w.float() - lr * grad.sign() * w.float().abs().mean()).bfloat16())
    return losses


def serve(block, lens=(70, 1, 200), steps=20, seed=2):
    """Prefill of packed prompts and decoding steps; the largest difference from the block run over the whole
    sequences, relative to the largest output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    S, width = len(lens), block.w_qkv.shape[1]
    whole = [torch.randn(n + steps, width, generator=g, device="cuda").bfloat16() for n in lens]
    offsets = lambda ns: torch.tensor([0, *torch.tensor(ns).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    cache = Cache(block, S, max(lens) + steps)
    cache.prefill(block, torch.cat([t[:n] for t, n in zip(whole, lens)])[None], offsets(lens))
    got = [cache.step(block, torch.stack([t[n + i] for t, n in zip(whole, lens)])) for i in range(steps)]
    ref, _ = block.forward(torch.cat(whole)[None], offsets([n + steps for n in lens]))
    at = offsets([n + steps for n in lens]).tolist()
    want = torch.stack([torch.stack([ref[0, at[s] + lens[s] + i] for s in range(S)]) for i in range(steps)]).float()
    return float((torch.stack(got).float() - want).abs().max() / want.abs().max())


def main():
    block = AttentionBlock()
    losses = train(block)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps", flush=True)
    print(f"serving: decoding differs from the whole prompt by {serve(block):.2e} of the largest output", flush=True)


if __name__ == "__main__":
    main()
