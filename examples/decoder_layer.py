#!/usr/bin/env python3
"""One decoder layer on the package's operators: a prompt in chunks, then tokens
one at a time, for several sequences that share a paged cache of 8 or 4 bits.

    python examples/decoder_layer.py [--seqs 4] [--prompt 300] [--chunk 128] [--tokens 8] [--bits 8]

The norms take the residual sum with them. Attention: norms of q and k for each head and
rotary positions in one pass, append to the cache, attention over it. FFN: the
predictor-gated sparse SwiGLU layer. The projections around them are plain matrix
products. Pages, positions and slots come from the GPU. Weights and inputs are random:
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
        """x: the layer's input after its norm."""
        T = x.shape[0]
        qkv = (x @ self.w_qkv.t()).view(T, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q, k = sffn.qk_norm_rope(q, k, positions, self.table, self.q_norm, self.k_norm)
        sffn.kv_cache_append(cache, batch, k, v)
        o = sffn.cache_attention(cache, batch, q, window=window)
        return o.view(T, -1) @ self.w_o.t()

    def __call__(self, x, positions, cache, batch, window=0):
        """x [T, d] of the batch's tokens at `positions`; their keys and values go
        into the cache."""
        y, _ = sffn.add_rms_norm(x, weight=self.norm1)
        y, x = sffn.add_rms_norm(self.attention(y, positions, cache, batch, window), x, self.norm2)
        return x + self.ffn(y)


class Sequences:
    """Block tables and lengths of sequences that grow together in one cache. The pages are
    handed out on the GPU as they are needed, here from a shuffled stack."""

    def __init__(self, n, layer, pages_each, page=64, bits=8):
        self.cache = (sffn.KVCache4 if bits == 4 else sffn.KVCache).empty(n * pages_each, layer.kv_heads,
                                                                          layer.head_dim, page)
        self.table = torch.full((n, pages_each), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.free, self.n_free = sffn.free_pages(n * pages_each)
        self.free = self.free[torch.randperm(n * pages_each, generator=torch.Generator().manual_seed(1)).cuda()]
        self.longest = [0] * n

    def extend(self, new):
        """Room for new[b] tokens more in sequence b: their positions and the batch."""
        self.longest = [have + m for have, m in zip(self.longest, new)]
        plan = sffn.page_plan(self.table, self.lens, torch.tensor(new, dtype=torch.int32, device="cuda"),
                              self.free, self.n_free, self.cache.page, sum(new))
        self.lens, self.n_free = plan.kv_lens, plan.n_free
        return plan.positions, sffn.CacheBatch(self.table, plan.kv_lens, max(self.longest), plan.cu, max(new),
                                               slots=plan.slots)


def run(layer, prompts, tokens, chunk, window=0, bits=8):
    """Prompts (a [n_b, d] tensor for each sequence) in chunks, then `tokens` steps
    that feed each sequence its last output. Returns every sequence's outputs."""
    n = len(prompts)
    pages = -(-(max(p.shape[0] for p in prompts) + tokens) // 64)
    seqs = Sequences(n, layer, pages, bits=bits)
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
    ap.add_argument("--bits", type=int, default=8, choices=(4, 8), help="bits of a cached channel")
    a = ap.parse_args()
    layer = DecoderLayer()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    prompts = [torch.randn(max(1, a.prompt - 37 * b), layer.d, generator=g, device="cuda").bfloat16()
               for b in range(a.seqs)]
    run(layer, prompts, 1, a.chunk, bits=a.bits)
    torch.cuda.synchronize()
    t = time.perf_counter()
    outs = run(layer, prompts, a.tokens, a.chunk, bits=a.bits)
    torch.cuda.synchronize()
    total = sum(o.shape[0] for o in outs)
    print(f"{a.seqs} sequences, {a.bits}-bit cache, {total} tokens through the layer in {(time.perf_counter() - t) * 1e3:.2f} ms; "
          f"last outputs' mean square {[round(o[-1].float().square().mean().item(), 3) for o in outs]}")


if __name__ == "__main__":
    main()
