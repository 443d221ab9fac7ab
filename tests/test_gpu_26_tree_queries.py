"""GPU: attention of trees whose query rows have a channel far larger than the others, every kernel of attention_int8_tree by
name against the fp64 oracle: what a row's other channels keep does not hang on which kernel the sizes choose.

Bounds, u = 2^-24. A row of queries is held in fp16 terms, scaled so that its largest element lies in [8, 16):
 * bf16, one term (11 bits, the smallest step 2^-24): elements of at least 2^-20 of the largest are exact, and all are here;
 * fp32, two terms: each of 11 bits, so off by 2^-22 of the element, or by half the smallest step, 2^-28 of the largest.
Sums over D channels of NT terms round NT D / 16 + 2 times, 2 u each, the factors and the maximum's subtraction 10 times. With B
= scale sum |q| |k| and C the largest logit,
   delta = scale sum (2^-22 |q| + 2^-28 max |q|) |k| [fp32] + (NT D / 8 + 4) u B + 10 u (C + 8).
For lse and output then as in test_gpu_22_attention_tree.py.
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import drafts as ref
from test_gpu_14_kv_cache_int8 import DTYPES, _ints, _offsets
from test_gpu_15_attention_int8 import _cache
from test_gpu_22_attention_tree import _trees
from test_gpu_24_tree_kernels import PLANS, _fits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HEADS, KV, BS, PREFIX, NODES = 4, 2, 32, [300, 70], [20, 9]


def _delta(x, k, scale, fp32):
    B, C = abs(scale) * (np.abs(k) @ np.abs(x)).max(), np.abs(scale * (k @ x)).max()
    held = abs(scale) * (np.abs(k) @ (2.0 ** -22 * np.abs(x) + 2.0 ** -28 * np.abs(x).max())).max() if fp32 else 0.0
    return held + ((2 if fp32 else 1) * len(x) / 8 + 4) * U * B + 10 * U * (C + 8)


def _large_channel(api, gpu, dim, dtype, factor):
    """Queries with one channel `factor` times larger, and a cache whose keys have codes of -1, 0 and 1 there."""
    lens = [p + n for p, n in zip(PREFIX, NODES)]
    cache, table, vals = _cache(api, lens, KV, dim, BS, gpu, dim + 1)
    channel = dim // 2 + 3
    cache.k[..., channel] = cache.k[..., channel].sign()
    codes, scales = cache.k.cpu().double(), cache.k_scales.cpu().double()
    for b, (k, _) in enumerate(vals):
        ids = table[b, np.arange(len(k)) // BS].astype(np.int64)
        k[..., channel] = (codes[ids, :, np.arange(len(k)) % BS, channel] * scales[ids]).numpy()
    gen = torch.Generator().manual_seed(dim)
    Q = 1.5 * torch.randn(sum(NODES), HEADS, dim, generator=gen)
    Q = torch.where(Q.abs() < 2.0 ** -7, 0.5, Q)      # 2^-20 of the largest, and more
    Q[..., channel] *= factor
    Q = Q.to(DTYPES[dtype]).to(gpu)
    trees = _trees(NODES, 3, 5)
    return Q, cache, [_ints(_offsets(NODES), gpu), _ints(lens, gpu), _ints(table, gpu), _ints(sum(trees, []), gpu)], vals, trees


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [30, 1000])
@pytest.mark.parametrize("plan,dim", [(p, d) for p in [None] + PLANS for d in (64, 128, 256) if p is None or _fits(p, d)])
def test_a_large_channel(gpu, plan, dim, factor, dtype):
    from post_int4_weight_amd import api
    announce(f"attention tree kernel={plan} dim={dim} {dtype}, one channel {factor} times larger")
    Q, cache, args, vals, trees = _large_channel(api, gpu, dim, dtype, factor)
    scale, fp32 = dim ** -0.5, dtype == "f32"
    if plan is None:      # the one that the sizes choose
        O, lse = api.attention_int8_tree(Q, cache, *args, return_lse=True)
    else:
        O, lse = api._test_attention_int8_tree(*plan, Q, cache, *args)
    torch.cuda.synchronize()
    q, o, got, first = to64(Q), to64(O), to64(lse), 0
    for (k, v), parents in zip(vals, trees):
        for i in range(len(parents)):
            keys = ref.keys_of(parents, i, len(k) - len(parents))
            for h in range(HEADS):
                x, g, N = q[first + i, h], h // (HEADS // KV), len(keys)
                want, wl, A, _, _ = ref.attend(x, k[keys, g], v[keys, g], scale)
                delta = _delta(x, k[keys, g], scale, fp32)
                assert abs(got[first + i, h] - wl) <= delta + (N / 16 + 24) * 2 * U + 2 * U * abs(wl) + 2.0 ** -20, (i, h)
                tol = A * (2 * (delta + 4 * U) + (2.0 ** -21 if fp32 else 2.0 ** -11) + (N / 16 + 24) * 2 * U)
                tol = tol + 2.0 ** -30 * np.abs(v[:, g]).max() * N + 16 * U * np.abs(want)
                if not fp32:
                    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
                assert np.all(np.abs(o[first + i, h] - want) <= tol), (i, h)
        first += len(parents)
