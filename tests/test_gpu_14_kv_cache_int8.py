"""GPU: the int8 key/value cache (kv_cache_write_int8, kv_cache_read_int8)
against the fp64 oracle (oracle/int8.py).

Bounds. Scales are fp32 by definition and equal. A code equals the oracle's
except where x / S lies within code_slack of a tie; a code recoded after a
growth of its block's scale is rint(c ratio) with ratio two roundings away from
S_old / S, so the same slack holds (two roundings at 127 steps). The oracle
marks the codes that came within the slack of a tie; all others are equal, and
those are off by one at most (a recoding's ratio is below 1).
Reading back multiplies code and scale in fp32: equal bit for bit.
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import int8 as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _table(lens, bs, num_blocks, seed, width=None):
    """Shuffled blocks for sequences of the given lengths; -1 past them."""
    rng = np.random.default_rng(seed)
    ids = rng.permutation(num_blocks)
    width = width or max(1, -(-max(lens) // bs))
    table, used = np.full((len(lens), width), -1, dtype=np.int32), 0
    for b, n in enumerate(lens):
        m = -(-n // bs)
        table[b, :m] = ids[used:used + m]
        used += m
    assert used <= num_blocks
    return table


def _ints(v, gpu):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=gpu)


def _offsets(n):
    return [0] + np.cumsum(n).tolist()


def _rows(total, heads, dim, dtype, gpu, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(total, heads, dim, generator=gen) * torch.exp(0.5 * torch.randn(total, 1, 1, generator=gen))
    return x.to(DTYPES[dtype]).to(gpu)


def _codes(cache):
    """Both halves as [num_blocks, heads, bs, dim]."""
    return {"k": cache.k.cpu().numpy().astype(np.int64),
            "v": cache.v.cpu().numpy().transpose(0, 1, 3, 2).astype(np.int64)}


def _check_codes(cache, want, table, lens):
    bs = want.bs
    got = _codes(cache)
    scales = {"k": to64(cache.k_scales), "v": to64(cache.v_scales)}
    for half in "kv":
        for b, n in enumerate(lens):
            for p0 in range(0, n, bs):
                i, m = table[b][p0 // bs], min(bs, n - p0)
                assert np.array_equal(scales[half][i], want.scales[half][i]), (half, b, p0)
                d = np.abs(got[half][i][:, :m] - want.codes[half][i][:, :m])
                assert np.all(d <= want.near[half][i][:, :m]), (half, b, p0, int(d.max()))


def _check_read(api, cache, offsets, starts, table, dtype, gpu):
    rows = offsets[-1]
    k, v = api.kv_cache_read_int8(cache, _ints(offsets, gpu), _ints(starts, gpu), _ints(table, gpu), rows,
                                  out_dtype=DTYPES[dtype])
    torch.cuda.synchronize()
    codes, bs = _codes(cache), cache.k.shape[2]
    for got, half, scales in ((k, "k", cache.k_scales.cpu().numpy()), (v, "v", cache.v_scales.cpu().numpy())):
        for b, start in enumerate(starts):
            for r in range(offsets[b], offsets[b + 1]):
                p = start + r - offsets[b]
                i = table[b][p // bs]
                x = codes[half][i][:, p % bs].astype(np.float32) * scales[i][:, None]
                assert torch.equal(got[r].cpu(), torch.from_numpy(x).to(DTYPES[dtype])), (half, b, p)


# per call, tokens that each sequence appends
HISTORIES = [[(5, 0, 1), (1, 1, 1), (1, 30, 0), (40, 3, 2)],
             [(16, 17, 128, 1), (0, 0, 0, 0), (1, 1, 1, 1), (130, 15, 31, 255)],
             [(3,)] + [(1,)] * 20]


@pytest.mark.parametrize("history", HISTORIES, ids=["short", "ragged", "appends"])
@pytest.mark.parametrize("heads,dim,bs,dtype", [(1, 64, 16, "bf16"), (3, 128, 16, "f32"), (2, 64, 32, "f32"),
                                                (2, 128, 64, "bf16"), (1, 256, 128, "bf16"), (2, 256, 16, "f32"),
                                                (1, 128, 128, "f32")])
def test_write_and_read(gpu, history, heads, dim, bs, dtype):
    from post_int4_weight_amd import api
    announce(f"kv cache heads={heads} dim={dim} bs={bs} {dtype} history={history[:3]}")
    lens = np.sum(history, axis=0).tolist()
    nb = sum(-(-n // bs) for n in lens) + 2
    table = _table(lens, bs, nb, seed=bs + dim)
    cache = api.KVCacheInt8.empty(nb, heads, dim, bs, device=gpu)
    cache.k.fill_(77)          # what was in the blocks before
    cache.v.fill_(-77)
    cache.k_scales.fill_(1e3)
    cache.v_scales.fill_(1e3)
    want = ref.Cache(nb, heads, dim, bs)
    starts = [0] * len(lens)
    for call, new in enumerate(history):
        off = _offsets(new)
        k, v = (_rows(off[-1], heads, dim, dtype, gpu, 100 * call + i) for i in (0, 1))
        api.kv_cache_write_int8(cache, k, v, _ints(off, gpu), _ints(starts, gpu), _ints(table, gpu))
        torch.cuda.synchronize()
        want.write("k", to64(k), off, starts, table)
        want.write("v", to64(v), off, starts, table)
        starts = [s + n for s, n in zip(starts, new)]
        _check_codes(cache, want, table, starts)
        # one call again: the same cache
        before = [t.clone() for t in cache]
        api.kv_cache_write_int8(cache, k, v, _ints(off, gpu), _ints([s - n for s, n in zip(starts, new)], gpu),
                                _ints(table, gpu))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cache, before))
    untouched = sorted(set(range(nb)) - set(table[table >= 0].tolist()))
    assert (cache.k[untouched] == 77).all() and (cache.v_scales[untouched] == 1e3).all()
    _check_read(api, cache, _offsets(lens), [0] * len(lens), table, dtype, gpu)
    # a range in the middle, and no rows of some sequences
    part = [max(0, n - 4) if b % 2 == 0 else 0 for b, n in enumerate(lens)]
    if sum(part):
        _check_read(api, cache, _offsets(part), [min(3, n - m) for n, m in zip(lens, part)], table, "bf16", gpu)


def test_many_sequences(gpu):
    """More sequences than a wave has lanes, empty ones among them."""
    from post_int4_weight_amd import api
    announce("kv cache, 150 sequences")
    lens = [(7 * b) % 5 + (40 if b % 50 == 3 else 0) for b in range(150)]
    bs, heads, dim = 16, 2, 64
    nb = sum(-(-n // bs) for n in lens)
    table, off = _table(lens, bs, nb, 9), _offsets(lens)
    cache = api.KVCacheInt8.empty(nb, heads, dim, bs, device=gpu)
    k, v = (_rows(off[-1], heads, dim, "bf16", gpu, i) for i in (1, 2))
    api.kv_cache_write_int8(cache, k, v, _ints(off, gpu), _ints([0] * 150, gpu), _ints(table, gpu))
    torch.cuda.synchronize()
    want = ref.Cache(nb, heads, dim, bs)
    want.write("k", to64(k), off, [0] * 150, table)
    want.write("v", to64(v), off, [0] * 150, table)
    _check_codes(cache, want, table, lens)
    _check_read(api, cache, off, [0] * 150, table, "f32", gpu)


def test_row_strides(gpu):
    """K and V are column ranges of one projection's output; read back into such ranges."""
    from post_int4_weight_amd import api
    announce("kv cache, strided rows")
    bs, heads, dim, n = 32, 2, 64, 45
    qkv = _rows(n, 3 * heads, dim, "bf16", gpu, 4)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    table = _table([n], bs, 4, 1)
    args = (_ints([0, n], gpu), _ints([0], gpu), _ints(table, gpu))
    a, b = (api.KVCacheInt8.empty(4, heads, dim, bs, device=gpu) for _ in range(2))
    api.kv_cache_write_int8(a, k, v, *args)
    api.kv_cache_write_int8(b, k.contiguous(), v.contiguous(), *args)
    wide = torch.full((n, 3 * heads, dim), 9.0, device=gpu)
    api.kv_cache_read_int8(a, *args, n, K=wide[:, :heads], V=wide[:, 2 * heads:])
    x, y = api.kv_cache_read_int8(b, *args, n, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert torch.equal(wide[:, :heads], x) and torch.equal(wide[:, 2 * heads:], y)
    assert (wide[:, heads:2 * heads] == 9.0).all()


def test_zero_and_non_finite(gpu):
    from post_int4_weight_amd import api
    announce("kv cache, zero, NaN and infinite values")
    bs, dim = 16, 64
    x = torch.randn(48, 2, dim, generator=torch.Generator().manual_seed(0)).to(gpu)
    x[0:16, 0] = 0
    x[20, 1, 3] = float("nan")
    x[40, 0, 60] = float("inf")
    cache = api.KVCacheInt8.empty(5, 2, dim, bs, device=gpu)
    table = _ints([[3, 0, 4]], gpu)
    api.kv_cache_write_int8(cache, x, x, _ints([0, 48], gpu), _ints([0], gpu), table)
    k, v = api.kv_cache_read_int8(cache, _ints([0, 48], gpu), _ints([0], gpu), table, 48, out_dtype=torch.float32)
    torch.cuda.synchronize()
    for y in (k, v):
        assert (y[:16, 0] == 0).all() and torch.isfinite(y[:16]).all()
        assert torch.isnan(y[16:32, 1]).all() and torch.isfinite(y[16:32, 0]).all()
        assert torch.isnan(y[32:, 0]).all() and torch.isfinite(y[32:, 1]).all()
    # the block stays NaN while it is appended to, and is clean when it starts again
    api.kv_cache_write_int8(cache, x[:1], x[:1], _ints([0, 1], gpu), _ints([31], gpu), table)
    assert torch.isnan(cache.k_scales[0, 1])
    api.kv_cache_write_int8(cache, x[:1], x[:1], _ints([0, 1], gpu), _ints([16], gpu), table)
    torch.cuda.synchronize()
    assert torch.isfinite(cache.k_scales[0]).all()


def test_positions_without_a_block(gpu):
    """Ids outside the pool, positions past the table and negative starts: not written, read as NaN."""
    from post_int4_weight_amd import api
    announce("kv cache, positions without a block")
    bs, dim, n = 16, 64, 80
    x = torch.randn(2 * n, 1, dim, generator=torch.Generator().manual_seed(0)).to(gpu)
    cache = api.KVCacheInt8.empty(6, 1, dim, bs, device=gpu)
    table = _ints([[0, 6, -1, 2], [3, 4, 5, 1]], gpu)       # 64 positions each
    args = (_ints([0, n, 2 * n], gpu), _ints([0, -5], gpu), table)
    api.kv_cache_write_int8(cache, x, x, *args)
    k, v = api.kv_cache_read_int8(cache, *args, 2 * n, out_dtype=torch.float32)
    torch.cuda.synchronize()
    for y in (k, v):
        bad = torch.isnan(y).all(2).all(1).cpu().numpy()
        want = np.ones(2 * n, dtype=bool)
        want[0:16] = want[48:64] = False
        assert np.array_equal(bad, want) and not torch.isnan(y[:16]).any()
    assert (cache.k_scales[[3, 4, 5, 1]] == 0).all()         # the second sequence wrote nothing
    # offsets that leave the rows are cut to them
    api.kv_cache_write_int8(cache, x, x, _ints([0, n, 10 ** 9], gpu), _ints([0, 0], gpu), table)
    torch.cuda.synchronize()
    assert (cache.k_scales[[3, 4, 5, 1]] > 0).all()


def test_large_cache(gpu):
    """Blocks whose codes lie more than 2^31 bytes into the pool."""
    from post_int4_weight_amd import api
    announce("kv cache of more than 2^32 codes")
    bs, heads, dim = 128, 8, 128
    nb = (1 << 32) // (bs * heads * dim) + 4
    cache = api.KVCacheInt8.empty(nb, heads, dim, bs, device=gpu)
    table = [[nb - 1, 1, nb - 2]]
    off, n = [0, 300], 300
    x = _rows(n, heads, dim, "bf16", gpu, 3)
    api.kv_cache_write_int8(cache, x, x, _ints(off, gpu), _ints([0], gpu), _ints(table, gpu))
    k, v = api.kv_cache_read_int8(cache, _ints(off, gpu), _ints([0], gpu), _ints(table, gpu), n, out_dtype=torch.float32)
    small = api.KVCacheInt8.empty(3, heads, dim, bs, device=gpu)
    t = _ints([[0, 1, 2]], gpu)
    api.kv_cache_write_int8(small, x, x, _ints(off, gpu), _ints([0], gpu), t)
    k0, v0 = api.kv_cache_read_int8(small, _ints(off, gpu), _ints([0], gpu), t, n, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(k, k0) and torch.equal(v, v0) and torch.equal(k, v)
    assert int(cache.k_scales.count_nonzero()) == 3 * heads


def test_refusals(gpu):
    from post_int4_weight_amd import api
    cache = api.KVCacheInt8.empty(4, 2, 64, 16, device=gpu)
    x = torch.ones(3, 2, 64, device=gpu)
    off, st, table = _ints([0, 3], gpu), _ints([0], gpu), _ints([[0]], gpu)
    with pytest.raises(ValueError):
        api.kv_cache_write_int8(cache, x[:, :1], x, off, st, table)
    with pytest.raises(ValueError):
        api.kv_cache_write_int8(cache, x, x, off.long(), st, table)
    with pytest.raises(ValueError):
        api.kv_cache_write_int8(cache, x, x, off, st, _ints([0], gpu))
    with pytest.raises(TypeError):
        api.kv_cache_write_int8(cache, x, x.bfloat16(), off, st, table)
    with pytest.raises(ValueError):
        api.kv_cache_write_int8(cache._replace(v=cache.k), x, x, off, st, table)
    with pytest.raises(api.PTQError) as e:
        odd = api.KVCacheInt8.empty(4, 2, 96, 16, device=gpu)
        y = torch.ones(3, 2, 96, device=gpu)
        api.kv_cache_write_int8(odd, y, y, off, st, table)
    assert e.value.name == "PTQ_EINVAL" and "head_dim" in str(e.value)
    with pytest.raises(api.PTQError):
        odd = api.KVCacheInt8.empty(4, 2, 64, 24, device=gpu)
        api.kv_cache_read_int8(odd, off, st, table, 3)
