"""GPU: rotary positions (rotary_apply) and appending with them (kv_cache_append_int8) against the fp64 oracle
(oracle/drafts.py).

Bound of a turned value, u = 2^-24: the reduced angle is rounded once (at most 2^-25) after fp64 work off by 2^-51 |t|; its
sine and cosine are Taylor sums whose last operations round twice, at most 4 u together; the magnitude, the two products and
their sum round once each: (|x_a| + |x_b|) m (8 u + 2^-51 |t|), then half a step of the output's type.
Appending is writing what rotary_apply gives in fp32: the same arithmetic, so the same bits.
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import drafts as ref
from test_gpu_14_kv_cache_int8 import DTYPES, _ints, _offsets, _rows, _table

pytestmark = pytest.mark.gpu


def _check(Y, X, positions, rotary, dtype):
    x, f, m = to64(X), rotary.inv_freq.cpu().numpy(), rotary.magnitude
    want, n = ref.turn(x, positions, f, m, rotary.interleaved), len(f)
    tol = np.zeros_like(want)
    t = np.abs(np.asarray(positions, np.float64)[:, None, None] * f)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if rotary.interleaved else (slice(0, n), slice(n, 2 * n))
    tol[..., a] = tol[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(m) * (8 * 2.0 ** -24 + 2.0 ** -51 * t)
    if dtype == "bf16":
        tol[..., :2 * n] += 2.0 ** -8 * (np.abs(want[..., :2 * n]) + tol[..., :2 * n]) + 2.0 ** -134
    got = to64(Y)
    assert np.array_equal(got[..., 2 * n:], x[..., 2 * n:])
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot", [(1, 1, 8, 2), (1, 5, 8, 8), (3, 2, 64, 64), (70, 3, 80, 32), (33, 9, 72, 48),
                                                (5, 7, 96, 54), (130, 1, 128, 126), (600, 33, 128, 128), (9, 4, 256, 64),
                                                (2, 2, 120, 112), (12000, 9, 128, 128), (12000, 9, 128, 90)])
def test_rotary(gpu, rows, heads, dim, rot, interleaved, dtype):
    from post_int4_weight_amd import api
    announce(f"rotary rows={rows} heads={heads} dim={dim} rot={rot} interleaved={interleaved} {dtype}")
    rotary = api.Rotary.make(rot, interleaved=interleaved, device=gpu)._replace(magnitude=1.25 if rows % 2 else 1.0)
    X = _rows(rows, heads, dim, dtype, gpu, rows + rot)
    rng = np.random.default_rng(rows)
    pos = rng.integers(-100, 200000, rows)
    pos[0] = 0 if rows > 1 else 2 ** 31 - 1
    Y = api.rotary_apply(X, rotary, _ints(pos, gpu))
    Z = X.clone()
    assert api.rotary_apply(Z, rotary, _ints(pos, gpu), Y=Z) is Z
    # rows of a wider projection's output, into such rows
    wide = torch.full((rows, heads + 2, dim), 7.0, dtype=X.dtype, device=gpu)
    wide[:, 1:-1] = X
    into = torch.full_like(wide, 9.0)
    api.rotary_apply(wide[:, 1:-1], rotary, _ints(pos, gpu), Y=into[:, 2:])
    torch.cuda.synchronize()
    _check(Y, X, pos, rotary, dtype)
    assert torch.equal(Z, Y) and torch.equal(into[:, 2:], Y) and (into[:, :2] == 9).all()


def test_far_positions_and_odd_frequencies(gpu):
    """Angles of up to 2^31 radians and more, of frequencies that no formula gives, zero among them."""
    from post_int4_weight_amd import api
    announce("rotary, far positions")
    f = torch.tensor([1.0, 0.0, 3.7, 1e-30, 0.5, 2.0 ** -31, 1e-3, 6.25], dtype=torch.float64, device=gpu)
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 1048576, 99]
    for il in (False, True):
        X = _rows(len(pos), 2, 64, "f32", gpu, 5)
        rotary = api.Rotary(f, 1.0, il)
        Y = api.rotary_apply(X, rotary, _ints(pos, gpu))
        torch.cuda.synchronize()
        _check(Y, X, pos, rotary, "f32")


def test_values_that_are_not_finite(gpu):
    """They reach their own pair and nothing else."""
    from post_int4_weight_amd import api
    announce("rotary, NaN and infinities")
    for il, rot in ((False, 32), (True, 30), (False, 30)):
        rotary = api.Rotary.make(rot, interleaved=il, device=gpu)
        X = _rows(6, 3, 64, "bf16", gpu, 1)
        clean = api.rotary_apply(X, rotary, _ints(range(6), gpu))
        X[2, 1, 3], X[4, 0, 40], X[5, 2, 31] = float("nan"), float("inf"), float("-inf")
        Y = api.rotary_apply(X, rotary, _ints(range(6), gpu))
        torch.cuda.synchronize()
        hit = torch.zeros_like(X, dtype=torch.bool)
        hit[2, 1, [3, 2 if il else 3 + rot // 2]] = True
        hit[4, 0, 40] = True
        hit[5, 2, [31] if rot == 30 else [31, 15]] = True
        assert torch.equal(Y[~hit], clean[~hit]) and not torch.isfinite(Y[hit]).any()
        assert Y[4, 0, 40] == float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved,rot", [(False, 64), (False, 32), (False, 22), (True, 64), (True, 6)])
@pytest.mark.parametrize("heads,dim,bs", [(1, 64, 16), (3, 64, 128), (2, 128, 32), (5, 128, 64), (2, 256, 16), (1, 256, 128)])
def test_append(gpu, heads, dim, bs, interleaved, rot, dtype):
    from post_int4_weight_amd import api
    rot = rot * dim // 64 if rot != 22 else rot
    announce(f"append heads={heads} dim={dim} bs={bs} rot={rot} interleaved={interleaved} {dtype}")
    rotary = api.Rotary.make(rot, interleaved=interleaved, device=gpu)
    history = [(5, 0, 1, 200), (1, 1, 1, 1), (1, 30, 0, 7), (40, 3, 2, 130)]
    lens = np.sum(history, axis=0).tolist()
    nb = sum(-(-n // bs) for n in lens) + 2
    table = _table(lens, bs, nb, seed=bs + dim)
    a, b = (api.KVCacheInt8.empty(nb, heads, dim, bs, device=gpu) for _ in range(2))
    for c in (a, b):      # what was in the blocks before
        c.k.fill_(77), c.v.fill_(-77), c.k_scales.fill_(1e3), c.v_scales.fill_(1e3)
    starts, far = [0] * len(lens), [0, 100000, 7, 50]
    for call, new in enumerate(history):
        off = _offsets(new)
        k, v = (_rows(off[-1], heads, dim, dtype, gpu, 100 * call + i) for i in (0, 1))
        pos = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, new)])
        given = call % 2 == 1      # positions of their own: shared ones among them, as in a tree
        if given:
            pos = np.repeat(far, new) + pos // 2
        args = (_ints(off, gpu), _ints(starts, gpu), _ints(table, gpu))
        api.kv_cache_append_int8(a, k, v, *args, rotary, positions=_ints(pos, gpu) if given else None)
        turned = api.rotary_apply(k.float(), rotary, _ints(pos, gpu))
        api.kv_cache_write_int8(b, turned, v.float(), *args)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b)), call
        starts = [s + n for s, n in zip(starts, new)]


def test_append_without_blocks_and_strides(gpu):
    """Positions without a block are not written, rows of no sequence do not matter, K and V may be column ranges."""
    from post_int4_weight_amd import api
    announce("append, positions without a block, strided rows")
    bs, dim, n = 16, 64, 80
    rotary = api.Rotary.make(dim, device=gpu)
    x = _rows(2 * n + 5, 3, dim, "f32", gpu, 0)
    a, b = (api.KVCacheInt8.empty(6, 1, dim, bs, device=gpu) for _ in range(2))
    args = (_ints([0, n, 2 * n], gpu), _ints([0, -5], gpu), _ints([[0, 6, -1, 2], [3, 4, 5, 1]], gpu))
    api.kv_cache_append_int8(a, x[:, :1], x[:, 2:], *args, rotary)
    turned = api.rotary_apply(x[:n, :1], rotary, _ints(range(n), gpu))
    api.kv_cache_write_int8(b, torch.cat([turned, x[n:, :1]]), x[:, 2:], *args)
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, b)) and (a.k_scales[[3, 4, 5, 1]] == 0).all() and (a.k_scales[0] > 0).all()
    # a NaN among the keys makes its block's scale NaN, not its neighbours'
    x[3, 0, 5] = float("nan")
    api.kv_cache_append_int8(a, x[:32, :1].contiguous(), x[:32, 2:].contiguous(), _ints([0, 32], gpu), _ints([0], gpu),
                             _ints([[0, 1]], gpu), rotary)
    torch.cuda.synchronize()
    assert torch.isnan(a.k_scales[0]).all() and torch.isfinite(a.k_scales[1]).all() and torch.isfinite(a.v_scales).all()
