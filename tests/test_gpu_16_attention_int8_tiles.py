"""attention_int8_cache where the work is enough for tiles of 256 rows (tables wide enough, or rows many enough, for that
choice): the same checks, with the same tolerances, as for few rows."""
import numpy as np
import pytest
import torch

from gpu_util import announce
from test_gpu_14_kv_cache_int8 import _ints, _offsets
from test_gpu_15_attention_int8 import _check, _run, _simple

pytestmark = pytest.mark.gpu
KEYS = 200_000       # that a row of the table has room for


def _wide(api, gpu, lens, qn, dtype="f32", **kw):
    bs = kw.get("bs", 16)
    cache, table, vals, Q, (off, ln, tb) = _simple(api, gpu, lens, qn, dtype, **kw)
    more = torch.full((len(lens), KEYS // bs - tb.shape[1]), -1, dtype=torch.int32, device=gpu)
    return cache, table, vals, Q, (off, ln, torch.cat([tb, more], 1).contiguous())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,bs", [(64, 16), (64, 32), (64, 64), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged(gpu, dim, bs, dtype, causal):
    """Lengths around the edges of blocks, steps and tiles; more queries than keys leaves rows empty."""
    from post_int4_weight_amd import api
    announce(f"attention tiles dim={dim} bs={bs} {dtype} causal={causal}")
    lens, qn = [130, 1, 300, 9, 0, 200, 64, 65, 191], [130, 1, 70, 20, 3, 0, 64, 33, 128]
    _run(api, gpu, lens, qn, 4, 2, dim, bs, dtype, causal=causal, seed=3, width=KEYS // bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim,bs", [(4, 4, 64, 16), (8, 2, 128, 64), (3, 1, 128, 16), (7, 1, 64, 128)])
def test_long(gpu, heads, kv, dim, bs, dtype):
    """Several steps without a mask, in one split and in many."""
    from post_int4_weight_amd import api
    announce(f"attention tiles, long prompts heads={heads}/{kv} dim={dim} bs={bs} {dtype}")
    _run(api, gpu, [700, 513, 1500], [700, 256, 333], heads, kv, dim, bs, dtype, seed=11, width=KEYS // bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [1, 37, 300])
def test_windows(gpu, dim, window, dtype):
    from post_int4_weight_amd import api
    announce(f"attention tiles, window {window} dim={dim} {dtype}")
    _run(api, gpu, [700, 900], [700, 640], 32, 1, dim, 64, dtype, window=window, seed=5, width=KEYS // 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_non_finite(gpu, dim, dtype):
    """S_v or S_k of a block that is not finite, blocks without a valid id: NaN to the rows that attend to them; S_v
    leaves lse as it was."""
    from post_int4_weight_amd import api
    announce(f"attention tiles, NaN blocks {dim} {dtype}")
    lens, qn = [700, 150], (300, 150)
    cache, table, vals, Q, (off, ln, tb) = _wide(api, gpu, lens, qn, dtype, dim=dim)
    clean, want = api.attention_int8_cache(Q, cache, off, ln, tb, return_lse=True)
    top = max(float(np.abs(v).max()) for _, v in vals)
    for at in (5, 9, 30, 42):                # positions 80 .. 95, 144 .., 480 .., 672 ..
        bad = int(table[0, at])
        seen = torch.zeros(Q.shape[:2], dtype=torch.bool, device=gpu)
        seen[:qn[0], 2:] = (torch.arange(lens[0] - qn[0], lens[0], device=gpu) >= 16 * at)[:, None]
        for which in ("v", "k", "id"):
            t2, scales = tb, cache.v_scales if which == "v" else cache.k_scales
            keep = scales[bad, 1].clone()
            if which == "id":
                t2 = tb.clone()
                t2[0, at] = cache.k.shape[0]
                seen[:qn[0], :2] = seen[:qn[0], 2:]
            else:
                scales[bad, 1] = float("nan")
            got, lse = api.attention_int8_cache(Q, cache, off, ln, t2, return_lse=True)
            torch.cuda.synchronize()
            scales[bad, 1] = keep
            assert torch.isnan(got[seen]).all(), (at, which)
            # the other rows' probabilities may be rounded against another reference: either answer is within
            # 2^-11 (2^-21) of sum w |v| <= top, and of its own rounding
            bits, out = (11, 8) if dtype == "bf16" else (21, 20)
            err = (got[~seen].double() - clean[~seen].double()).abs()
            assert (err <= 2.0 ** (1 - bits) * top + 2.0 ** (1 - out) * clean[~seen].double().abs()).all(), (at, which)
            ok = torch.ones_like(seen) if which == "v" else ~seen
            assert torch.allclose(lse[ok], want[ok], rtol=1e-5, atol=1e-5) and torch.isnan(lse[~ok]).all()


def test_zero_scales(gpu):
    from post_int4_weight_amd import api
    announce("attention tiles, zero blocks")
    for dtype in ("f32", "bf16"):
        cache, table, vals, Q, args = _wide(api, gpu, [350], (120,), dtype)
        k, v = (x.copy() for x in vals[0])
        for blocks in (range(0, 2), range(4, 7), range(0, 22)):
            ids = table[0, list(blocks)].astype(np.int64)
            cache.v_scales[ids] = 0.0
            cache.k_scales[ids] = 0.0
            for i in blocks:
                k[16 * i:16 * i + 16] = 0
                v[16 * i:16 * i + 16] = 0
            O, lse = api.attention_int8_cache(Q, cache, *args, return_lse=True)
            torch.cuda.synchronize()
            _check(O, lse, Q, [(k, v)], (120,), 4, 2, 64, 64 ** -0.5, True, 0)


def test_uneven_scales(gpu):
    """Blocks of V many orders of magnitude apart, in either order: those that matter keep their bits."""
    from post_int4_weight_amd import api
    announce("attention tiles, scales of V that rise and fall")
    for dtype in ("f32", "bf16"):
        cache, table, vals, Q, args = _wide(api, gpu, [640], (200,), dtype, dim=128)
        ids = table[0].astype(np.int64)
        for order in (range(40), range(39, -1, -1)):
            k, v = (x.copy() for x in vals[0])
            keep = cache.v_scales.clone()
            for i, blk in enumerate(order):
                cache.v_scales[ids[blk]] *= 2.0 ** i
                v[16 * blk:16 * blk + 16] *= 2.0 ** i
            O, lse = api.attention_int8_cache(Q, cache, *args, return_lse=True)
            torch.cuda.synchronize()
            # an absolute error of the largest value a row attends to is all that a sum can keep
            o, q = O.double().cpu().numpy(), Q.double().cpu().numpy()
            for h in range(4):
                g = h // 2
                s = q[:, h] @ k[:, g].T / 128 ** 0.5
                s[np.arange(640)[None] > (440 + np.arange(200))[:, None]] = -np.inf
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                top = np.where(np.isfinite(s), np.abs(v[:, g]).max(1)[None], 0).max(1)
                err = np.abs(o[:, h] - w @ v[:, g])
                # probabilities of 11 bits (22) and a bf16 (fp32) result
                assert np.all(err <= top[:, None] * (2.0 ** -7 if dtype == "bf16" else 2.0 ** -15)), (dtype, h)
            cache.v_scales.copy_(keep)


def test_graph_and_streams(gpu):
    from post_int4_weight_amd import api
    announce("attention tiles, another stream, graph replays")
    qn = (320, 133)
    cache, table, vals, Q, args = _wide(api, gpu, [900, 333], qn, dtype="bf16", dim=128)
    want = api.attention_int8_cache(Q, cache, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = api.attention_int8_cache(Q * 1.0, cache, *args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    q, O = torch.zeros_like(Q), torch.empty_like(Q)
    need = api.attention_int8_cache_workspace_bytes(sum(qn), 2, 4, 2, 128, 16, args[2].shape[1])
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
    from test_gpu_15_attention_int8 import _cache
    announce("attention tiles over a cache of more than 2^32 codes")
    bs, heads, dim = 128, 8, 128
    nb = (1 << 32) // (bs * heads * dim) + 4
    big = api.KVCacheInt8.empty(nb, heads, dim, bs, device=gpu)
    small, table, vals = _cache(api, [300], heads, dim, bs, gpu, 2)
    far = [nb - 1, 0, nb - 2]
    for s, t in zip(small, big):
        t[far] = s[table[0].astype(np.int64)]
    wide = lambda ids: _ints([list(ids) + [-1] * (KEYS // bs)], gpu)
    Q = torch.randn(200, 16, dim, generator=torch.Generator().manual_seed(1)).bfloat16().to(gpu)
    a = api.attention_int8_cache(Q, small, _ints(_offsets([200]), gpu), _ints([300], gpu), wide(table[0]))
    b = api.attention_int8_cache(Q, big, _ints(_offsets([200]), gpu), _ints([300], gpu), wide(far))
    torch.cuda.synchronize()
    assert torch.equal(a, b)
