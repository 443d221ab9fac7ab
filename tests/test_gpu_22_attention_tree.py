"""GPU: attention of trees of drafted tokens (attention_int8_tree) against the fp64 oracle (oracle/drafts.py) on the values
that the cache's codes stand for.

Bounds, per output element, u = 2^-24 and A = sum w |v| / sum w:
 * a logit: q is a whole number of steps, at most 1 / 16256 (bf16) or 1 / 2080768 (fp32) of its row's largest element |q|_max;
   rounding to one is off by half a step, and by 2^-23 of the largest number before that: 0.502 or 0.75 of a step. The sum
   over channels is exact. Its conversion, the factors, the maximum's subtraction: 10 roundings of a logit C (and of the
   shift by 8): delta = step scale sum|k| + 10 u (C + 8).
 * a probability: off by delta and 4 u for the exponential; in fp16 2^-11 (bf16 queries) or 2^-21 (two terms); S_v against
   its running maximum 4 u.
 * the sum over N keys: N / 16 matrix steps and 24 more roundings, 2 u each; the joins 16 u.
 * the smallest fp16 step against the largest probability: 2^-30 of the largest value a key.
so |err| <= A (2 (delta + 4 u) + P + (N / 16 + 24) 2 u) + 2^-30 top N + 16 u |o| + half a step of the output's type.
lse: delta + (N / 16 + 24) 2 u + 2 u |lse| + 2^-20.
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import drafts as ref
from test_gpu_14_kv_cache_int8 import DTYPES, _ints, _offsets
from test_gpu_15_attention_int8 import _cache

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _trees(nodes, reach, seed):
    """Parents of each sequence's nodes, below one of the `reach` before them or nothing."""
    rng = np.random.default_rng(seed)
    return [[int(max(-1, i - 1 - rng.integers(0, reach))) for i in range(n)] for n in nodes]


def _check(O, lse, Q, vals, trees, heads, kv, scale, window):
    q, o, got, first = to64(Q), to64(O), to64(lse), 0
    fp32, worst = Q.dtype == torch.float32, 0.0
    for (k, v), parents in zip(vals, trees):
        n = len(parents)
        base = k.shape[0] - n
        for i in range(n):
            keys = ref.keys_of(parents, i, base, window)
            for h in range(heads):
                if keys is None:
                    assert np.isnan(o[first + i, h]).all() and np.isnan(got[first + i, h])
                    continue
                x, g, N = q[first + i, h], h // (heads // kv), len(keys)
                want, wl, A, _, C = ref.attend(x, k[keys, g], v[keys, g], scale)
                step = np.abs(x).max() * (0.75 / 2080768 if fp32 else 0.502 / 16256)
                delta = step * abs(scale) * np.abs(k[keys, g]).sum(1).max() + 10 * U * (C + 8)
                tol = A * (2 * (delta + 4 * U) + (2.0 ** -21 if fp32 else 2.0 ** -11) + (N / 16 + 24) * 2 * U)
                tol = tol + 2.0 ** -30 * np.abs(v[:, g]).max() * N + 16 * U * np.abs(want)
                if not fp32:
                    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
                err = np.abs(o[first + i, h] - want)
                assert np.all(err <= tol), (i, h, float((err / tol).max()))
                worst = max(worst, float((err / tol).max()))
                tl = delta + (N / 16 + 24) * 2 * U + 2 * U * abs(wl) + 2.0 ** -20
                assert abs(got[first + i, h] - wl) <= tl, (i, h, got[first + i, h], wl)
        first += n


def _make(api, gpu, prefix, trees, heads, kv, dim, bs, dtype, seed=0, width=None):
    nodes = [len(t) for t in trees]
    lens = [p + n for p, n in zip(prefix, nodes)]
    cache, table, vals = _cache(api, lens, kv, dim, bs, gpu, seed, width)
    gen = torch.Generator().manual_seed(seed + 1)
    Q = (1.5 * torch.randn(sum(nodes), heads, dim, generator=gen)).to(DTYPES[dtype]).to(gpu)
    flat = _ints([p for t in trees for p in t], gpu)
    return Q, cache, [_ints(_offsets(nodes), gpu), _ints(lens, gpu), _ints(table, gpu), flat], vals


def _run(api, gpu, prefix, trees, heads, kv, dim, bs, dtype, window=0, scale=None, seed=0, width=None):
    Q, cache, args, vals = _make(api, gpu, prefix, trees, heads, kv, dim, bs, dtype, seed, width)
    O, lse = api.attention_int8_tree(Q, cache, *args, scale=scale, window=window, return_lse=True)
    again = api.attention_int8_tree(Q, cache, *args, scale=scale, window=window)
    torch.cuda.synchronize()
    _check(O, lse, Q, vals, trees, heads, kv, scale or dim ** -0.5, window)
    assert torch.equal(O, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,bs", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (256, 16), (256, 64)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2), (6, 2), (8, 1)])
def test_small_trees(gpu, heads, kv, dim, bs, dtype):
    """Trees that start and end inside blocks and steps, single tokens, no tokens, no keys before the tree."""
    from post_int4_weight_amd import api
    announce(f"attention tree heads={heads}/{kv} dim={dim} bs={bs} {dtype}")
    prefix, nodes = [0, 0, 63, 64, 50, 127, 9, 300, 15], [1, 7, 1, 2, 20, 0, 5, 33, 17]
    _run(api, gpu, prefix, _trees(nodes, 4, dim + bs), heads, kv, dim, bs, dtype, seed=dim + bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 3, 40, 130, 1000, 2 ** 62])
def test_windows(gpu, window, dim, dtype):
    from post_int4_weight_amd import api
    announce(f"attention tree window={window} dim={dim} {dtype}")
    _run(api, gpu, [130, 0, 61, 500], _trees([40, 30, 1, 12], 3, window % 97), 4, 2, dim, 32, dtype, window=window, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim,reach", [(2, 2, 64, 1), (4, 1, 128, 6), (8, 1, 64, 3), (2, 1, 256, 9), (3, 1, 128, 600)])
def test_large_trees(gpu, heads, kv, dim, reach, dtype):
    """Up to the largest, chains (reach 1) and bushes; several tiles of rows each, waves without rows."""
    from post_int4_weight_amd import api
    announce(f"attention tree large heads={heads}/{kv} dim={dim} reach={reach} {dtype}")
    _run(api, gpu, [33, 500], _trees([512, 70], reach, reach), heads, kv, dim, 64, dtype, seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes,heads", [(3, 4), (12, 4), (25, 4), (40, 8), (1, 1)])
def test_long_keys(gpu, nodes, heads, dtype):
    """Split keys, one tile of each size and more; and a table far wider than its sequences."""
    from post_int4_weight_amd import api
    announce(f"attention tree nodes={nodes} heads={heads} over long keys {dtype}")
    _run(api, gpu, [5000, 20], _trees([nodes, 2], 3, 1), heads, 1, 128, 64, dtype, seed=21)
    _run(api, gpu, [3000], _trees([nodes], 2, 2), heads, 1, 64, 16, dtype, seed=22, width=3000)
    _run(api, gpu, [2500, 10], _trees([nodes, 4], 2, 3), heads, 1, 128, 32, dtype, window=1100, seed=23)


def test_scales(gpu):
    from post_int4_weight_amd import api
    announce("attention tree, softmax scales")
    for scale in (1e-6, -0.2, 1.0):
        for dtype in DTYPES:
            _run(api, gpu, [90, 7], _trees([9, 30], 4, 8), 2, 1, 64, 16, dtype, scale=scale, seed=31)


def test_many_sequences(gpu):
    from post_int4_weight_amd import api
    announce("attention tree, 150 sequences")
    nodes = [(7 * b) % 5 + (20 if b % 50 == 3 else 0) for b in range(150)]
    _run(api, gpu, [(13 * b) % 70 for b in range(150)], _trees(nodes, 2, 9), 2, 2, 64, 16, "bf16", seed=41)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chain_is_causal_attention(gpu, dtype):
    """A chain of tokens gives what attention_int8_cache does, within both bounds."""
    from post_int4_weight_amd import api
    announce(f"attention tree, a chain {dtype}")
    trees = [list(range(-1, n - 1)) for n in (50, 3, 200)]
    Q, cache, args, vals = _make(api, gpu, [100, 700, 0], trees, 6, 2, 128, 32, dtype, 51)
    O, lse = api.attention_int8_tree(Q, cache, *args, return_lse=True)
    P, other = api.attention_int8_cache(Q, cache, *args[:3], return_lse=True)
    torch.cuda.synchronize()
    _check(O, lse, Q, vals, trees, 6, 2, 128 ** -0.5, 0)
    near = 2e-2 if dtype == "bf16" else 2e-5
    assert torch.allclose(O.float(), P.float(), rtol=near, atol=near) and torch.allclose(lse, other, rtol=1e-3, atol=1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_trees_and_lengths(gpu, dtype):
    """What a parent that is not below its node, a tree longer than its sequence or than 512, a sequence longer than the
    table and a block without an id give: NaN to the rows concerned, nothing to the others."""
    from post_int4_weight_amd import api
    announce(f"attention tree, bad trees and lengths {dtype}")
    good = _trees([20, 20, 20, 20], 3, 1)
    Q, cache, args, vals = _make(api, gpu, [700, 30, 100, 10], good, 4, 2, 64, 16, dtype, 61)
    want, wl = api.attention_int8_tree(Q, cache, *args, return_lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all()
    for at, value in ((5, 5), (5, 19), (0, 3), (9, -2), (11, 2 ** 31 - 1), (3, 513), (3, -2 ** 31)):
        flat = args[3].clone()
        flat[20 + at] = value
        bad = [list(t) for t in good]
        bad[1][at] = value
        O, lse = api.attention_int8_tree(Q, cache, *args[:3], flat, return_lse=True)
        torch.cuda.synchronize()
        hit = torch.tensor([i // 20 == 1 and ref.line(bad[1], i - 20) is None for i in range(80)], device=gpu)
        assert hit.any() and torch.isnan(O[hit]).all() and torch.isnan(lse[hit]).all()
        assert torch.equal(O[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])
    for lens in ([720, 19, 120, 30], [10 ** 6, 50, 120, 30], [720, -7, 120, 30], [720, 0, 120, 30]):
        O = api.attention_int8_tree(Q, cache, args[0], _ints(lens, gpu), *args[2:])
        torch.cuda.synchronize()
        hit = torch.tensor([lens[i // 20] not in (720, 50, 120, 30) for i in range(80)], device=gpu)
        assert torch.isnan(O[hit]).all() and torch.equal(O[~hit], want[~hit])
    table = args[2].clone()      # sequence 2: positions 100 .. 119 are the tree, in blocks 6 and 7
    table[2, 7] = 10 ** 6
    O = api.attention_int8_tree(Q, cache, *args[:2], table, args[3])
    torch.cuda.synchronize()
    hit = torch.tensor([i // 20 == 2 and any(100 + x >= 112 for x in ref.line(good[2], i - 40)) if i // 20 == 2 else False
                        for i in range(80)], device=gpu)
    assert hit.any() and torch.isnan(O[hit]).all() and torch.equal(O[~hit], want[~hit])
    # 513 nodes
    Q, cache, args, _ = _make(api, gpu, [10, 3], _trees([513, 4], 3, 2), 1, 1, 64, 16, dtype, 62)
    O = api.attention_int8_tree(Q, cache, *args)
    torch.cuda.synchronize()
    assert torch.isnan(O[:513]).all() and torch.isfinite(O[513:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_of_blocks_not_attended(gpu, dim, dtype):
    """Blocks before a window and nodes of other branches may hold anything: NaN, infinite or huge scales of theirs leave a
    row's bits alone. Ones that it attends to make O NaN, and lse only if S_k is."""
    from post_int4_weight_amd import api
    announce(f"attention tree, scales of blocks not attended {dim} {dtype}")
    # nodes 0 .. 15 in one block, 16 .. 31 in the next; the latter hang below node 3 or 20
    parents = [-1] + [i // 2 for i in range(15)] + [3 if i % 2 else 20 for i in range(16)]
    parents[16:21] = [3] * 5
    Q, cache, args, vals = _make(api, gpu, [64], [parents], 4, 2, dim, 16, dtype, 71)
    for window, first in ((0, None), (12, 0)):
        want, wl = api.attention_int8_tree(Q, cache, *args, window=window, return_lse=True)
        torch.cuda.synchronize()
        assert torch.isfinite(want).all()
        for block, hit in ((5, list(range(16, 32))), (0, [] if window else list(range(32)))):
            hit = torch.tensor([i in hit for i in range(32)], device=gpu)
            at = int(args[2][0, block])
            for value in (float("nan"), float("inf"), 1e30):
                for scales in (cache.k_scales, cache.v_scales):
                    keep = scales[at].clone()
                    scales[at] = value
                    O, lse = api.attention_int8_tree(Q, cache, *args, window=window, return_lse=True)
                    torch.cuda.synchronize()
                    scales[at] = keep
                    assert torch.equal(O[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit]), (window, block, value)
                    if value != 1e30:
                        assert torch.isnan(O[hit]).all()
                    if scales is cache.v_scales:
                        assert torch.allclose(lse, wl, rtol=1e-5, atol=1e-5)


def test_queries_that_are_zero_or_not_finite(gpu):
    from post_int4_weight_amd import api
    announce("attention tree, zero, tiny, NaN and infinite queries")
    trees = _trees([40], 3, 4)
    for dtype in DTYPES:
        Q, cache, args, vals = _make(api, gpu, [90], trees, 2, 1, 64, 16, dtype, 81)
        Q[3], Q[4, 1] = 0, Q[4, 1] * 1e-36
        O, lse = api.attention_int8_tree(Q, cache, *args, return_lse=True)
        torch.cuda.synchronize()
        _check(O, lse, Q, vals, trees, 2, 1, 0.125, 0)
        X = Q.clone()
        X[7, 0, 5], X[9, 1, 63] = float("nan"), float("-inf")
        P = api.attention_int8_tree(X, cache, *args)
        torch.cuda.synchronize()
        hit = torch.zeros(40, 2, dtype=torch.bool, device=gpu)
        hit[7, 0] = hit[9, 1] = True
        assert torch.isnan(P[hit]).all() and torch.equal(P[~hit], O[~hit])


def test_strides_and_rows_of_no_sequence(gpu):
    from post_int4_weight_amd import api
    announce("attention tree, strided rows, rows behind the last sequence")
    trees = _trees([12, 9], 3, 6)
    for prefix, width in (([90, 40], None), ([3000, 40], None)):      # without splits and with them
        Q, cache, args, vals = _make(api, gpu, prefix, trees, 4, 2, 64, 16, "bf16", 91, width)
        want, wl = api.attention_int8_tree(Q, cache, *args, return_lse=True)
        wide = torch.full((30, 12, 64), 5.0, dtype=Q.dtype, device=gpu)
        wide[:21, 4:8] = Q
        into, lse = torch.full_like(wide, 9.0), torch.full((30, 4), 9.0, device=gpu)
        more = torch.cat([args[3], torch.full((9,), 10 ** 9, dtype=torch.int32, device=gpu)])
        api.attention_int8_tree(wide[:, 4:8], cache, *args[:3], more, O=into[:, 2:6], lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(into[:21, 2:6], want) and torch.equal(lse[:21], wl)
        assert (into[21:] == 9).all() and (into[:, :2] == 9).all() and (into[:, 6:] == 9).all() and (lse[21:] == 9).all()


def test_streams_and_graphs(gpu):
    """On a stream of its own; captured with another call that shares its workspace, and replayed on new inputs."""
    from post_int4_weight_amd import api
    announce("attention tree, streams and graphs")
    trees = _trees([24, 10], 3, 7)
    made = [_make(api, gpu, [3000, 100], trees, 8, 2, 128, 64, "bf16", s) for s in (1, 2)]
    want = [api.attention_int8_tree(Q, c, *a) for Q, c, a, _ in made]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = api.attention_int8_tree(made[0][0], made[0][1], *made[0][2])
    side.synchronize()
    assert torch.equal(got, want[0])
    q, c = made[0][0].clone(), api.KVCacheInt8(*(t.clone() for t in made[0][1]))
    args = [t.clone() for t in made[0][2]]
    need = api.attention_int8_tree_workspace_bytes(34, 2, 8, 2, 128, api.PTQ_BF16, 64, args[2].shape[1])
    assert need > 0
    ws, O1, O2 = torch.empty(need, dtype=torch.uint8, device=gpu), torch.empty_like(q), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.attention_int8_tree(q, c, *args, O=O1, workspace=ws)
        api.attention_int8_tree(q, c, *args, O=O2, workspace=ws, window=500)
    for i in (0, 1, 0, 1):
        q.copy_(made[i][0])
        for x, y in zip(c, made[i][1]):
            x.copy_(y)
        args[2].copy_(made[i][2][2])
        O1.zero_(), ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O1, want[i])
        assert torch.equal(O2, api.attention_int8_tree(*made[i][:2], *made[i][2], window=500)) and not torch.equal(O1, O2)


def test_large_pool(gpu):
    """Blocks whose codes lie more than 2^32 bytes into the pool."""
    from post_int4_weight_amd import api
    announce("attention tree over a pool of more than 2^32 codes")
    trees = _trees([20], 3, 8)
    Q, cache, args, _ = _make(api, gpu, [300], trees, 16, 8, 128, 128, "bf16", 3)
    want = api.attention_int8_tree(Q, cache, *args)
    nb = (1 << 32) // (128 * 8 * 128) + 4
    big = api.KVCacheInt8.empty(nb, 8, 128, 128, device=gpu)
    ids = torch.tensor([nb - 1, 1, nb - 2], device=gpu)
    old = args[2][0, :3].long()
    for x, y in zip(big, cache):
        x[ids] = y[old]
    got = api.attention_int8_tree(Q, big, *args[:2], ids.int()[None], args[3])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
