#!/usr/bin/env python3
"""A transformer block over sparse voxels: training steps, then decoding from a cache.

The voxels of several objects are ordered along the Morton curve of their hash,
object after object, and embedded by a submanifold convolution. The block is
norm and rotation of the queries and keys by the voxels' own coordinates
(qk_norm_rope), attention in a window along that order with a few sink tokens
(window_attention), and a projection with a residual. Gradients come from
window_attention_backward, qk_norm_rope_backward, backward_data and
backward_weights. `decode` then runs the trained block causally over one object,
a prompt first and then token by token against its key-value cache.

    python examples/voxel_transformer.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import submanifold_sparse_conv_amd as sc
from gen import workloads


class SparseConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, kmap):
        ctx.save_for_backward(x, w)
        ctx.kmap = kmap
        return sc.forward(kmap, x, w)

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dy = dy.contiguous()
        dx = sc.backward_data(ctx.kmap, dy, sc.pack_weights_dgrad(w)) if ctx.needs_input_grad[0] else None
        return dx, sc.backward_weights(ctx.kmap, x, dy).to(w.dtype), None


class NormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_gain, k_gain, pos, freqs):
        ctx.save_for_backward(q, k, q_gain, k_gain, pos, freqs)
        return sc.qk_norm_rope(q, k, pos, freqs, q_gain, k_gain)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, q_gain, k_gain, pos, freqs = ctx.saved_tensors
        return (*sc.qk_norm_rope_backward(dq, dk, q, k, pos, freqs, q_gain, k_gain), None, None)


class WindowAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, window):
        out, lse = sc.window_attention(q, k, v, return_lse=True, **window)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.window = window
        return out

    @staticmethod
    def backward(ctx, dout):
        return (*sc.window_attention_backward(dout, *ctx.saved_tensors, **ctx.window), None)


class Block(torch.nn.Module):
    """Convolution, then attention with `heads` query heads and `kv_heads` key-value heads."""

    def __init__(self, c_in=64, width=128, heads=4, kv_heads=2, dim=32, window=64, sinks=4, device="cuda"):
        super().__init__()
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.left, self.sinks = window, sinks
        kw = dict(dtype=torch.bfloat16, device=device)

        def weight(*shape, fan):
            return torch.nn.Parameter(torch.randn(*shape, **kw) * fan ** -0.5)

        self.conv = weight(27, c_in, width, fan=9 * c_in)
        self.qkv = weight(width, (heads + 2 * kv_heads) * dim, fan=width)
        self.proj = weight(heads * dim, width, fan=heads * dim)
        self.q_gain = torch.nn.Parameter(torch.ones(heads, dim, device=device))
        self.k_gain = torch.nn.Parameter(torch.ones(kv_heads, dim, device=device))
        self.register_buffer("freqs", sc.rope_frequencies(dim, axes=3, device=device))

    def rotated(self, t, pos):
        """Rotated queries and keys, and the values, of the tokens t [n, width]."""
        qkv = (t @ self.qkv).view(t.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        return (*NormRope.apply(q, k, self.q_gain, self.k_gain, pos, self.freqs), v)

    def forward(self, x, kmap, pos, cu, causal=False):
        t = SparseConv.apply(x, self.conv, kmap)
        q, k, v = self.rotated(t, pos)
        window = dict(cu_q=cu, cu_k=cu, left=self.left, right=0 if causal else self.left, sinks=self.sinks)
        o = WindowAttention.apply(q, k, v, window)
        return t + o.flatten(1) @ self.proj

    @torch.no_grad()
    def decode(self, t, pos, prompt):
        """The block's causal output for the embedded tokens t of one object: the
        first `prompt` in one call, the rest one at a time against the cache."""
        n, dev = t.shape[0], t.device
        keys, values = (torch.empty(n, self.kv_heads, self.dim, dtype=t.dtype, device=dev) for _ in range(2))
        cu_k = torch.tensor([0, n], dtype=torch.int32, device=dev)
        outs, at = [], 0
        while at < n:
            m = prompt if at == 0 else 1
            q, k, v = self.rotated(t[at:at + m], pos[at:at + m])
            keys[at:at + m], values[at:at + m] = k, v
            at += m
            o = sc.window_attention(q, keys, values, cu_q=torch.tensor([0, m], dtype=torch.int32, device=dev), cu_k=cu_k,
                                    k_len=torch.tensor([at], dtype=torch.int32, device=dev), left=self.left, right=0,
                                    sinks=self.sinks)
            outs.append(t[at - m:at] + o.flatten(1) @ self.proj)
        return torch.cat(outs)


def voxels(objects=2, device="cuda"):
    """Coordinates (b, x, y, z) of `objects` 64^3 objects in Morton order, their
    kernel map and the token offsets of each object."""
    parts = []
    for b in range(objects):
        c = torch.from_numpy(workloads.make("S", seed_offset=b).coords).clone()
        c[:, 0] = b
        parts.append(c)
    coords = torch.cat(parts).to(device=device, dtype=torch.int32).contiguous()
    rows = sc.hash_sorted_rows(sc.build_hash(coords, grid_log2=6, batch=objects)).long()
    coords = coords[rows].contiguous()
    h = sc.build_hash(coords, grid_log2=6, batch=objects)
    counts = torch.bincount(coords[:, 0].long(), minlength=objects)
    cu = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
    return coords, sc.build_kernel_map(h), cu


def train(steps=20, objects=2, lr=2e-3, seed=0):
    """Fits the block to a fixed random target; returns (block, losses, x, coords, map, offsets)."""
    torch.manual_seed(seed)
    coords, kmap, cu = voxels(objects)
    block = Block()
    x = torch.randn(coords.shape[0], 64, dtype=torch.bfloat16, device="cuda")
    with torch.no_grad():
        teacher = Block()
        target = teacher(x, kmap, coords[:, 1:], cu).float()
    opt = torch.optim.Adam(block.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        loss = (block(x, kmap, coords[:, 1:], cu).float() - target).square().mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return block, torch.stack(losses).tolist(), x, coords, kmap, cu


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args(argv)
    block, losses, x, coords, kmap, cu = train(args.steps)
    print(f"{coords.shape[0]} voxels, loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    with torch.no_grad():
        n = min(256, int(cu[1]))
        t = sc.forward(kmap, x, block.conv.detach())[:n]
        out = block.decode(t, coords[:n, 1:], prompt=n - 64)
    print(f"decoded 64 tokens after a prompt of {n - 64}: output {tuple(out.shape)}, rms {out.float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
