"""An attention layer in 8 bits, from calibration to decoding.

    python examples/attention_layer_int8.py

A random attention layer of hidden size 1024 (8 query heads on 2 kv heads of 128 channels) is quantized with GPTQ to
8-bit codes with one scale per output channel, and then serves three sequences: their prompts in one ragged call, then
single tokens. Each step is linear_int8 for q, k and v, kv_cache_write_int8, attention_int8_cache and linear_int8 for o;
the outputs are compared with the same layer in fp32.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import post_int4_weight_amd as ptq  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, BLOCK = 1024, 8, 2, 128, 64


def quantize(W, X):
    """GPTQ codes of W [out, in] for inputs like X: 8 bits, one group per output channel."""
    n = W.shape[1]
    H, d = torch.zeros(n, n, device=W.device), torch.zeros(n, dtype=torch.float64, device=W.device)
    ptq.hessian_accumulate(H, d, X)
    layer = ptq.gptq_quantize_layer(W, H, d, bits=8, group_size=n)
    return layer["codes"], layer["scales"].flatten()


class AttentionInt8:
    """Projections in int8 codes, and a cache of `blocks` blocks that sequences take as they grow."""

    def __init__(self, weights, calibration, blocks=64):
        self.q, self.k, self.v = (quantize(weights[name], calibration) for name in "qkv")
        self.o = quantize(weights["o"], reference(weights, [calibration])[1])
        self.cache = ptq.KVCacheInt8.empty(blocks, KV_HEADS, DIM, BLOCK, device=calibration.device)
        self.free, self.tables, self.lengths = list(range(blocks)), [], []

    def step(self, tokens):
        """The next tokens of each sequence (a list of [n, HIDDEN], n >= 0); their outputs, in one ragged batch."""
        device = self.cache.k.device
        while len(self.tables) < len(tokens):
            self.tables.append([])
            self.lengths.append(0)
        starts = list(self.lengths)
        for b, x in enumerate(tokens):
            self.lengths[b] += x.shape[0]
            while len(self.tables[b]) * BLOCK < self.lengths[b]:
                self.tables[b].append(self.free.pop())
        width = max(len(t) for t in self.tables)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
        table = ints([t + [-1] * (width - len(t)) for t in self.tables])
        offsets = ints([0] + [x.shape[0] for x in tokens]).cumsum(0, dtype=torch.int32)
        X = torch.cat(tokens)
        rows = X.shape[0]
        q = ptq.linear_int8(X, *self.q).view(rows, HEADS, DIM)
        k = ptq.linear_int8(X, *self.k).view(rows, KV_HEADS, DIM)
        v = ptq.linear_int8(X, *self.v).view(rows, KV_HEADS, DIM)
        ptq.kv_cache_write_int8(self.cache, k, v, offsets, ints(starts), table)
        a = ptq.attention_int8_cache(q, self.cache, offsets, ints(self.lengths), table)
        return ptq.linear_int8(a.view(rows, HEADS * DIM), *self.o).split([x.shape[0] for x in tokens])


def reference(weights, sequences):
    """The layer in fp32 over whole sequences: outputs, and the o projection's inputs (bf16, all rows)."""
    outs, mixed = [], []
    for x in sequences:
        n, y = x.shape[0], x.float()
        q = (y @ weights["q"].float().T).view(n, KV_HEADS, HEADS // KV_HEADS, DIM).permute(1, 2, 0, 3)
        k = (y @ weights["k"].float().T).view(n, KV_HEADS, 1, DIM).permute(1, 2, 0, 3)
        v = (y @ weights["v"].float().T).view(n, KV_HEADS, 1, DIM).permute(1, 2, 0, 3)
        s = q @ k.transpose(-1, -2).contiguous() * DIM ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -torch.inf)
        a = (s.softmax(-1) @ v).permute(2, 0, 1, 3).reshape(n, HEADS * DIM)
        mixed.append(a)
        outs.append(a @ weights["o"].float().T)
    return outs, torch.cat(mixed).bfloat16()


def run(device="cuda", prompts=(700, 33, 250), decoded=40, seed=0):
    """Relative errors (Frobenius) of the prompts' outputs and of the decoded tokens' against fp32."""
    gen = torch.Generator().manual_seed(seed)
    draw = lambda *shape: torch.randn(*shape, generator=gen)
    out = {"q": HEADS * DIM, "k": KV_HEADS * DIM, "v": KV_HEADS * DIM, "o": HIDDEN}
    weights = {name: (draw(n, HIDDEN) / HIDDEN ** 0.5).bfloat16().to(device) for name, n in out.items()}
    sequences = [draw(n + decoded, HIDDEN).bfloat16().to(device) for n in prompts]
    layer = AttentionInt8(weights, draw(4096, HIDDEN).bfloat16().to(device))
    got = [[y] for y in layer.step([x[:n] for x, n in zip(sequences, prompts)])]
    for i in range(decoded):
        for ys, y in zip(got, layer.step([x[n + i:n + i + 1] for x, n in zip(sequences, prompts)])):
            ys.append(y)
    want, _ = reference(weights, sequences)
    error = lambda a, b: float((a - b).norm() / b.norm())
    first = error(torch.cat([y[0].float() for y in got]), torch.cat([w[:n] for w, n in zip(want, prompts)]))
    later = error(torch.cat([torch.cat(y[1:]).float() for y in got]),
                  torch.cat([w[n:] for w, n in zip(want, prompts)]))
    return first, later


if __name__ == "__main__":
    first, later = run()
    print(f"relative error against fp32: prompts {first:.4f}, decoded tokens {later:.4f}")
