"""GPU: attention over the int8 cache (attention_int8_cache) against the fp64
oracle (oracle/int8.py) on the values the cache's codes stand for.

Bounds, per output element, u = 2^-24 (fp32) and A = sum w |v| / sum w:
 * a logit: sum_d |q k| scale =: B is summed in fp32 by 13 roundings at most on
   its way through 32-deep matrix steps (5 levels inside one, 8 steps at 256
   channels), each at most 2u; q of two fp16 terms is 2^-22 off; the factors
   S_k, the softmax scale and the maximum's subtraction round the logit C three
   times in units of log2 e: delta = 32 u B + 6 u (C + 8) + 2^-22 B [fp32 q].
   A probability is then off by delta, and by 4u for the exponential.
 * a probability in fp16: 2^-11 (bf16 queries), or 2^-21 in two terms.
 * the sum over N keys: N / 32 matrix steps and 16 more roundings, 2u each.
 * V's scale against its running maximum: two roundings.
 * the output: 2^-8 |o| for bf16 (8 significant bits), and the join of the waves and splits, 16 u.
so |err| <= A (2 (delta + 4u) + P + (N / 32 + 24) 2u) + out, P = 2^-11 or 2^-21,
plus the smallest fp16 step against the largest probability, 2^-25 2^-8 A0, A0
the largest |v| of the row's keys times N / sum w <= N: below 2^-30 A0 N.
lse: delta + (N / 16 + 24) 2u + 2u |lse| + 2^-20.
"""
import math

import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import int8 as ref
from test_gpu_14_kv_cache_int8 import DTYPES, _ints, _offsets, _table

pytestmark = pytest.mark.gpu
U = ref.U


def _cache(api, lens, heads, dim, bs, gpu, seed, width=None):
    """A cache of normal codes with scales of uneven blocks, and its values [seq][half] -> [len, heads, dim]."""
    gen = torch.Generator().manual_seed(seed)
    nb = sum(-(-n // bs) for n in lens) + 3
    table = _table(lens, bs, nb, seed, width)
    code = lambda *s: (torch.randn(s, generator=gen) * 40).round().clamp(-128, 127).to(torch.int8)
    scale = lambda x: x * torch.exp(torch.randn(nb, heads, generator=gen))
    c = api.KVCacheInt8(code(nb, heads, bs, dim), code(nb, heads, dim, bs), scale(0.02), scale(0.01))
    vals = []
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // bs)].astype(np.int64)
        k = c.k[ids].double() * c.k_scales[ids].double()[..., None, None]
        v = c.v[ids].double() * c.v_scales[ids].double()[..., None, None]
        vals.append((k.permute(0, 2, 1, 3).reshape(-1, heads, dim)[:n].numpy(),
                     v.permute(0, 3, 1, 2).reshape(-1, heads, dim)[:n].numpy()))
    return api.KVCacheInt8(*(t.to(gpu) for t in c)), table, vals


def _check(O, lse, Q, vals, qn, heads, kv, dim, scale, causal, window, rows=None):
    q, o, got = to64(Q), to64(O), to64(lse)
    fp32 = Q.dtype == torch.float32
    first, worst, worst_l = 0, 0.0, 0.0
    for b, n in enumerate(qn):
        k, v = vals[b]
        length = k.shape[0]
        for h in range(heads):
            g = h // (heads // kv)
            if n == 0:
                continue
            want, wl, A, B, C, N = ref.attention(q[first:first + n, h], k[:, g], v[:, g], scale, length - n, causal, window)
            delta = 32 * U * B + 6 * U * (C + 8) + (2.0 ** -22 * B if fp32 else 0)
            top = np.abs(v[:, g]).max() if length else 0.0
            tol = A * (2 * (delta + 4 * U) + (2.0 ** -21 if fp32 else 2.0 ** -11) + (N / 32 + 24) * 2 * U)[:, None]
            tol = tol + (2.0 ** -30 * top * N)[:, None] + 16 * U * np.abs(want)
            if not fp32:
                tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
            err = np.abs(o[first:first + n, h] - want)
            assert np.all(err <= tol), (b, h, float((err - tol).max()), float((err / np.maximum(tol, 1e-30)).max()))
            worst = max(worst, float((err / np.maximum(tol, 1e-30)).max()))
            x = got[first:first + n, h]
            empty = np.isinf(wl)
            assert np.array_equal(np.isneginf(x), empty) and np.all(o[first:first + n, h][empty] == 0)
            tl = delta + (N / 16 + 24) * 2 * U + 2 * U * np.abs(wl) + 2.0 ** -20
            assert np.all(np.abs(x - wl)[~empty] <= tl[~empty]), (b, h)
        first += n


def _run(api, gpu, lens, qn, heads, kv, dim, bs, dtype, causal=True, window=0, scale=None, seed=0, width=None):
    cache, table, vals = _cache(api, lens, kv, dim, bs, gpu, seed, width)
    Q = (1.5 * torch.randn(sum(qn), heads, dim, generator=torch.Generator().manual_seed(seed + 1))).to(DTYPES[dtype]).to(gpu)
    args = (_ints(_offsets(qn), gpu), _ints(lens, gpu), _ints(table, gpu))
    kw = dict(scale=scale, causal=causal, window=window)
    O, lse = api.attention_int8_cache(Q, cache, *args, return_lse=True, **kw)
    again = api.attention_int8_cache(Q, cache, *args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(O, again)
    _check(O, lse, Q, vals, qn, heads, kv, dim, scale or dim ** -0.5, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,bs", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (256, 16), (256, 64)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2), (6, 2), (8, 1)])
def test_decode(gpu, heads, kv, dim, bs, dtype):
    """One query token; lengths around the edges of blocks and steps, empty ones among them."""
    from post_int4_weight_amd import api
    announce(f"attention decode heads={heads}/{kv} dim={dim} bs={bs} {dtype}")
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 130, 257, 700]
    _run(api, gpu, lens, [1] * len(lens), heads, kv, dim, bs, dtype, seed=dim + bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 37), (True, 200), (False, 0)])
def test_prompts(gpu, dim, dtype, causal, window):
    """Many query tokens, with and without earlier keys; more queries than keys leaves rows empty."""
    from post_int4_weight_amd import api
    announce(f"attention prompts dim={dim} {dtype} causal={causal} window={window}")
    lens, qn = [130, 1, 300, 9, 0, 200], [130, 1, 70, 20, 3, 0]
    _run(api, gpu, lens, qn, 4, 2, dim, 32, dtype, causal=causal, window=window, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim,bs", [(4, 4, 64, 16), (8, 2, 128, 64), (3, 1, 128, 16), (7, 1, 64, 128),
                                             (2, 1, 256, 32)])
def test_long_prompts(gpu, heads, kv, dim, bs, dtype):
    from post_int4_weight_amd import api
    announce(f"attention long prompts heads={heads}/{kv} dim={dim} bs={bs} {dtype}")
    _run(api, gpu, [700, 513, 400], [700, 256, 333], heads, kv, dim, bs, dtype, seed=11)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_speculated_tokens_and_long_keys(gpu, dtype):
    from post_int4_weight_amd import api
    announce(f"attention, a few query tokens over long keys {dtype}")
    _run(api, gpu, [5000, 20, 3001], [5, 3, 4], 8, 2, 128, 64, dtype, seed=21)
    _run(api, gpu, [9000], [1], 4, 1, 64, 16, dtype, seed=22, width=5000)     # a table far wider than the sequence
    _run(api, gpu, [4000, 10], [2, 2], 4, 4, 128, 32, dtype, window=100, seed=23)


def test_scales(gpu):
    """Softmax scales of other sizes and signs."""
    from post_int4_weight_amd import api
    announce("attention, softmax scales")
    for scale in (1e-6, -0.2, 1.0):
        _run(api, gpu, [90, 200], [1, 150], 2, 1, 64, 16, "f32", scale=scale, seed=31)


def _simple(api, gpu, lens, qn, dtype="f32", kv=2, heads=4, dim=64, bs=16, seed=5):
    cache, table, vals = _cache(api, lens, kv, dim, bs, gpu, seed)
    Q = torch.randn(sum(qn), heads, dim, generator=torch.Generator().manual_seed(seed)).to(DTYPES[dtype]).to(gpu)
    return cache, table, vals, Q, (_ints(_offsets(qn), gpu), _ints(lens, gpu), _ints(table, gpu))


@pytest.mark.parametrize("qn", [(1, 1), (2, 40), (150, 180)])
def test_non_finite_stays_with_its_rows(gpu, qn):
    """A NaN block is seen by the rows that attend to it only; NaN and infinite queries stay with their rows; rows of
    the pool that no length covers may hold anything."""
    from post_int4_weight_amd import api
    announce(f"attention, NaN blocks and queries {qn}")
    lens = [200, 181]
    cache, table, vals, Q, args = _simple(api, gpu, lens, qn)
    clean = api.attention_int8_cache(Q, cache, *args)
    torch.cuda.synchronize()
    # unused blocks, and everything past the table entries
    spare = sorted(set(range(cache.k.shape[0])) - set(table[table >= 0].tolist()))
    cache.k_scales[spare] = float("nan")
    cache.v_scales[spare] = float("inf")
    got = api.attention_int8_cache(Q, cache, *args)
    torch.cuda.synchronize()
    assert torch.equal(got, clean)
    # block 11 of sequence 0 (positions 176 .. 191): only queries from position 176 on see it
    bad = int(table[0, 11])
    for scales in (cache.k_scales, cache.v_scales):
        keep = scales[bad, 1].clone()
        scales[bad, 1] = float("nan")
        got = api.attention_int8_cache(Q, cache, *args)
        torch.cuda.synchronize()
        n = qn[0]
        seen = torch.arange(lens[0] - n, lens[0], device=gpu) >= 176
        assert torch.isnan(got[:n][seen][:, 2:]).all()            # heads 2, 3 read kv head 1
        rest = torch.cat([got[:n][~seen].flatten(), got[:n][:, :2].flatten(), got[n:].flatten()])
        same = torch.cat([clean[:n][~seen].flatten(), clean[:n][:, :2].flatten(), clean[n:].flatten()])
        assert torch.isfinite(rest).all()
        assert torch.allclose(rest, same, rtol=1e-5, atol=1e-6)
        scales[bad, 1] = keep
    Q2 = Q.clone()
    Q2[0, 0, 5] = float("nan")
    Q2[-1, 3, 9] = float("inf")
    got = api.attention_int8_cache(Q2, cache, *args)
    torch.cuda.synchronize()
    assert torch.isnan(got[0, 0]).all() and torch.isnan(got[-1, 3]).all()
    keep = torch.ones(Q.shape[:2], dtype=torch.bool, device=gpu)
    keep[0, 0] = keep[-1, 3] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("qn", [(1, 1), (300, 150)])
def test_non_finite_values_keep_lse(gpu, qn, dim, dtype):
    """S_v that is not finite makes the outputs NaN and leaves lse, which V has no part in, as it was."""
    from post_int4_weight_amd import api
    announce(f"attention, lse next to NaN values {qn} {dim} {dtype}")
    lens = [700, 150]
    cache, table, vals, Q, args = _simple(api, gpu, lens, qn, dtype, dim=dim)
    clean, want = api.attention_int8_cache(Q, cache, *args, return_lse=True)
    for at in (5, 42):                       # positions 80 .. 95, that all see; 672 .. 687
        bad = int(table[0, at])
        keep = cache.v_scales[bad, 1].clone()
        cache.v_scales[bad, 1] = float("nan")
        got, lse = api.attention_int8_cache(Q, cache, *args, return_lse=True)
        torch.cuda.synchronize()
        cache.v_scales[bad, 1] = keep
        seen = torch.zeros(Q.shape[:2], dtype=torch.bool, device=gpu)
        seen[:qn[0], 2:] = (torch.arange(lens[0] - qn[0], lens[0], device=gpu) >= 16 * at)[:, None]
        assert torch.isnan(got[seen]).all()
        assert torch.allclose(got[~seen].float(), clean[~seen].float(), rtol=2.0 ** -7, atol=1e-5)
        assert torch.allclose(lse, want, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("qn", [(1, 1), (100, 60)])
def test_bad_tables_and_lengths(gpu, qn):
    """Ids outside the pool give NaN; so does a length past the table, to its sequence only."""
    from post_int4_weight_amd import api
    announce(f"attention, ids and lengths out of range {qn}")
    lens = [100, 60]
    cache, table, vals, Q, (off, ln, tb) = _simple(api, gpu, lens, qn)
    clean = api.attention_int8_cache(Q, cache, off, ln, tb)
    for wrong in (cache.k.shape[0], -1, 2 ** 31 - 1):
        t2 = tb.clone()
        t2[1, 3] = wrong                                # positions 48 .. 63 of sequence 1
        got = api.attention_int8_cache(Q, cache, off, ln, t2)
        torch.cuda.synchronize()
        n = qn[0]
        seen = torch.arange(lens[1] - qn[1], lens[1], device=gpu) >= 48
        assert torch.equal(got[:n], clean[:n]) and torch.isnan(got[n:][seen]).all()
        assert torch.isfinite(got[n:][~seen]).all()
    got = api.attention_int8_cache(Q, cache, off, _ints([100, 2 ** 31 - 1], gpu), tb)
    torch.cuda.synchronize()
    assert torch.equal(got[:qn[0]], clean[:qn[0]]) and torch.isnan(got[qn[0]:]).all()
    got = api.attention_int8_cache(Q, cache, off, _ints([100, -7], gpu), tb)
    torch.cuda.synchronize()
    assert torch.equal(got[:qn[0]], clean[:qn[0]]) and (got[qn[0]:] == 0).all()


def test_zero_scales(gpu):
    """Blocks of zeros (scale 0), the first ones and all of them."""
    from post_int4_weight_amd import api
    announce("attention, zero blocks")
    for qn in ((1,), (120,)):
        cache, table, vals, Q, args = _simple(api, gpu, [150], qn)
        k, v = (x.copy() for x in vals[0])
        for blocks in (range(0, 2), range(4, 7), range(0, 10)):
            ids = table[0, list(blocks)].astype(np.int64)
            cache.v_scales[ids] = 0.0
            cache.k_scales[ids] = 0.0
            for i in blocks:
                k[16 * i:16 * i + 16] = 0
                v[16 * i:16 * i + 16] = 0
            O, lse = api.attention_int8_cache(Q, cache, *args, return_lse=True)
            torch.cuda.synchronize()
            _check(O, lse, Q, [(k, v)], qn, 4, 2, 64, 64 ** -0.5, True, 0)


def test_strides_streams_and_graphs(gpu):
    from post_int4_weight_amd import api
    announce("attention, strided rows, another stream, graph replays")
    for qn in ((1, 1), (120, 33)):
        cache, table, vals, Q, args = _simple(api, gpu, [900, 333], qn, dtype="bf16")
        want = api.attention_int8_cache(Q, cache, *args)
        wide = torch.randn(sum(qn), 12, 64, device=gpu).bfloat16()
        wide[:, 4:8] = Q
        out = torch.full_like(wide, 3.0)
        api.attention_int8_cache(wide[:, 4:8], cache, *args, O=out[:, 8:])
        torch.cuda.synchronize()
        assert torch.equal(out[:, 8:], want) and (out[:, :8] == 3.0).all()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = api.attention_int8_cache(Q * 1.0, cache, *args)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        q, O = torch.zeros_like(Q), torch.empty_like(Q)
        need = api.attention_int8_cache_workspace_bytes(sum(qn), 2, 4, 2, 64, 16, table.shape[1])
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=gpu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.attention_int8_cache(q, cache, *args, O=O, workspace=ws)
        for k in range(4):
            q.copy_(Q * (k + 1))
            graph.replay()
            got = O.clone()
            want = api.attention_int8_cache(q, cache, *args)
            torch.cuda.synchronize()
            assert torch.equal(got, want), k


def test_large_cache(gpu):
    """Blocks whose codes lie more than 2^32 bytes into the pool."""
    from post_int4_weight_amd import api
    announce("attention over a cache of more than 2^32 codes")
    bs, heads, dim = 128, 8, 128
    nb = (1 << 32) // (bs * heads * dim) + 4
    big = api.KVCacheInt8.empty(nb, heads, dim, bs, device=gpu)
    small, table, vals = _cache(api, [300], heads, dim, bs, gpu, 2)
    far = [nb - 1, 0, nb - 2]
    for s, t in zip(small, big):
        t[far] = s[table[0].astype(np.int64)]
    for n in (1, 200):
        Q = torch.randn(n, 16, dim, generator=torch.Generator().manual_seed(1)).bfloat16().to(gpu)
        a = api.attention_int8_cache(Q, small, _ints([0, n], gpu), _ints([300], gpu), _ints(table, gpu))
        b = api.attention_int8_cache(Q, big, _ints([0, n], gpu), _ints([300], gpu), _ints([far], gpu))
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_refusals(gpu):
    from post_int4_weight_amd import api
    cache, table, vals, Q, args = _simple(api, gpu, [40], (1,))
    with pytest.raises(api.PTQError) as e:
        api.attention_int8_cache(Q[:, :3], cache, *args)                 # 3 heads on 2 kv heads
    assert e.value.name == "PTQ_EINVAL" and "heads" in str(e.value)
    with pytest.raises(api.PTQError):
        api.attention_int8_cache(Q, cache, *args, scale=math.inf)
    with pytest.raises(api.PTQError):
        api.attention_int8_cache(Q, cache, *args, window=-1)
    with pytest.raises(api.PTQError):
        api.attention_int8_cache(Q, cache, *args, causal=False, window=4)
    with pytest.raises(TypeError):
        api.attention_int8_cache(Q.half(), cache, *args)
    with pytest.raises(ValueError):
        api.attention_int8_cache(Q[..., :32], cache, *args)
    need = api.attention_int8_cache_workspace_bytes(1, 1, 4, 2, 64, 16, 1000)
    assert need > 0
    with pytest.raises(api.PTQError) as e:
        api.attention_int8_cache(Q, cache, args[0], args[1], _ints(np.zeros((1, 1000)), gpu),
                                 workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
    assert e.value.name == "PTQ_EWORKSPACE"
