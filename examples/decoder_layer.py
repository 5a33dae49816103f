#!/usr/bin/env python3
"""One decoder layer on the package's operators: a prompt in chunks, then tokens
one at a time, for several sequences that share a paged 8-bit cache.

    python examples/decoder_layer.py [--seqs 4] [--prompt 300] [--chunk 128] [--tokens 8]

Attention: norms of q and k for each head and rotary positions in one pass, append
to the cache, attention over it. FFN: the predictor-gated sparse SwiGLU layer. The
projections around them are plain matrix products. Weights and inputs are random:
the layer's shapes are what is shown, not a trained model.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_sparse_ffn_amd as sffn  # noqa: E402


def rms_norm(x, weight, eps=1e-6):
    n = x.float()
    return (n * torch.rsqrt(n.square().mean(-1, keepdim=True) + eps)).to(x.dtype) * weight


class DecoderLayer:
    """Weights of one layer, bf16 on the GPU."""

    def __init__(self, d=1024, heads=8, kv_heads=2, head_dim=128, d_i=4096, rank=64, max_pos=4096, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).bfloat16()

        self.heads, self.kv_heads, self.head_dim, self.d = heads, kv_heads, head_dim, d
        self.w_qkv = weight((heads + 2 * kv_heads) * head_dim, d)
        self.w_o = weight(d, heads * head_dim)
        one = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        self.q_norm, self.k_norm = one, one.clone()
        self.norm1 = torch.ones(d, dtype=torch.bfloat16, device="cuda")
        self.norm2 = self.norm1.clone()
        # positions of a context four times the trained one
        self.table = sffn.rope_table(max_pos, head_dim, scaling="by_parts", factor=4.0, original_max_pos=max_pos // 4)
        self.ffn = sffn.SparseFFN(weight(d_i, d), weight(d_i, d), weight(d, d_i), weight(rank, d), weight(d_i, rank))

    def attention(self, x, positions, cache, batch, window=0):
        T = x.shape[0]
        qkv = (rms_norm(x, self.norm1) @ self.w_qkv.t()).view(T, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q, k = sffn.qk_norm_rope(q, k, positions, self.table, self.q_norm, self.k_norm)
        sffn.kv_cache_append(cache, batch, k, v)
        o = sffn.cache_attention(cache, batch, q, window=window)
        return o.view(T, -1) @ self.w_o.t()

    def __call__(self, x, positions, cache, batch, window=0):
        """x [T, d] of the batch's tokens at `positions`; their keys and values go
        into the cache."""
        x = x + self.attention(x, positions, cache, batch, window)
        return x + self.ffn(rms_norm(x, self.norm2))


class Sequences:
    """Block tables and lengths of sequences that grow together in one cache. Pages
    are handed out as they are needed, in no order of the sequences."""

    def __init__(self, n, layer, pages_each, page=64):
        self.n, self.page = n, page
        self.cache = sffn.KVCache.empty(n * pages_each, layer.kv_heads, layer.head_dim, page)
        self.table = torch.zeros(n, pages_each, dtype=torch.int32)
        self.lens = [0] * n
        self.used = [0] * n
        self.free = torch.randperm(n * pages_each, generator=torch.Generator().manual_seed(1)).tolist()

    def extend(self, new):
        """Room for new[b] tokens more in sequence b: their positions and the batch."""
        positions = []
        for b, m in enumerate(new):
            positions += range(self.lens[b], self.lens[b] + m)
            self.lens[b] += m
            while self.used[b] * self.page < self.lens[b]:
                self.table[b, self.used[b]] = self.free.pop()
                self.used[b] += 1
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = sffn.CacheBatch(self.table.cuda(), torch.tensor(self.lens, **i32), max(self.lens),
                                torch.tensor(cu, **i32), max(new))
        return torch.tensor(positions, **i32), batch


def run(layer, prompts, tokens, chunk, window=0):
    """Prompts (a [n_b, d] tensor for each sequence) in chunks, then `tokens` steps
    that feed each sequence its last output. Returns every sequence's outputs."""
    n = len(prompts)
    pages = -(-(max(p.shape[0] for p in prompts) + tokens) // 64)
    seqs = Sequences(n, layer, pages)
    outs = [[] for _ in range(n)]

    def step(xs):
        positions, batch = seqs.extend([x.shape[0] for x in xs])
        y = layer(torch.cat(xs), positions, seqs.cache, batch, window)
        for b, part in enumerate(y.split([x.shape[0] for x in xs])):
            if part.shape[0]:
                outs[b].append(part)

    longest = max(p.shape[0] for p in prompts)
    for at in range(0, longest, chunk):
        step([p[at:at + chunk] for p in prompts])       # sequences whose prompt has ended wait
    for _ in range(tokens):
        step([o[-1][-1:] for o in outs])
    return [torch.cat(o) for o in outs]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--chunk", type=int, default=128)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    layer = DecoderLayer()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    prompts = [torch.randn(max(1, a.prompt - 37 * b), layer.d, generator=g, device="cuda").bfloat16()
               for b in range(a.seqs)]
    run(layer, prompts, 1, a.chunk)
    torch.cuda.synchronize()
    t = time.perf_counter()
    outs = run(layer, prompts, a.tokens, a.chunk)
    torch.cuda.synchronize()
    total = sum(o.shape[0] for o in outs)
    print(f"{a.seqs} sequences, {total} tokens through the layer in {(time.perf_counter() - t) * 1e3:.2f} ms; "
          f"last outputs' mean square {[round(o[-1].float().square().mean().item(), 3) for o in outs]}")


if __name__ == "__main__":
    main()
