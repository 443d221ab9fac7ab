"""GPU: every kernel of attention_int8_tree by name (the hook in include/ptq_testing.h), with and without splits, against the
fp64 oracle within the bounds of test_gpu_22_attention_tree.py, which reaches the ones that the estimates choose."""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import drafts as ref
from test_gpu_22_attention_tree import _check, _make, _trees

pytestmark = pytest.mark.gpu

PLANS = [(0, 4, 1), (0, 4, 5), (0, 8, 1), (0, 8, 3), (1, 8, 1), (1, 8, 3), (2, 4, 1), (2, 4, 3), (2, 8, 1), (2, 8, 2)]      # tiles, waves, splits
SHAPES = [(64, 16), (64, 64), (128, 16), (128, 128), (256, 16), (256, 32)]


def _fits(plan, dim):
    return dim <= 128 or plan[1] == 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("plan,dim,bs", [(p, d, b) for p in PLANS for d, b in SHAPES if _fits(p, d)])
def test_kernel(gpu, plan, dim, bs, window, dtype):
    from post_int4_weight_amd import api
    announce(f"attention tree kernel={plan} dim={dim} bs={bs} window={window} {dtype}")
    # trees over the edges of steps, blocks and tiles; single nodes, no nodes, no keys before the tree
    prefix, nodes = [1000, 0, 250, 63, 31, 129], [45, 70, 1, 0, 17, 3]
    trees = _trees(nodes, 4, dim + window)
    Q, cache, args, vals = _make(api, gpu, prefix, trees, 6, 2, dim, bs, dtype, 7)
    O, lse = api._test_attention_int8_tree(*plan, Q, cache, *args, window=window)
    again, _ = api._test_attention_int8_tree(*plan, Q, cache, *args, window=window)
    torch.cuda.synchronize()
    _check(O, lse, Q, vals, trees, 6, 2, dim ** -0.5, window)
    assert torch.equal(O, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("plan,dim", [(p, d) for p in PLANS for d in (64, 128, 256) if _fits(p, d)])
def test_rows_by_themselves(gpu, plan, dim, dtype):
    """NaN queries, bad parents, scales that are not finite or huge: they reach the rows that see them, and no bit of others."""
    from post_int4_weight_amd import api
    announce(f"attention tree kernel={plan} dim={dim} {dtype}, rows by themselves")
    parents = [-1] + [i // 2 for i in range(15)] + [3] * 16      # two blocks of the cache
    Q, cache, args, _ = _make(api, gpu, [496, 80], [parents, parents[:16]], 4, 2, dim, 16, dtype, 9)
    run = lambda q=Q, flat=args[3]: api._test_attention_int8_tree(*plan, q, cache, *args[:3], flat)
    want, wl = run()
    torch.cuda.synchronize()
    assert torch.isfinite(want).all()

    def others(hit, got):
        hit = hit[:, None].expand(48, 4) if hit.dim() == 1 else hit
        assert torch.isnan(got[0][hit]).all() and torch.equal(got[0][~hit], want[~hit]) and torch.equal(got[1][~hit], wl[~hit])
    hit = torch.zeros(48, 4, dtype=torch.bool, device=gpu)
    q = Q.clone()
    q[5, 2, 7], q[40, 0, 0] = float("nan"), float("inf")
    hit[5, 2] = hit[40, 0] = True
    others(hit, run(q=q))
    flat = args[3].clone()
    flat[8] = 8      # and no node hangs below it
    others(torch.arange(48, device=gpu) == 8, run(flat=flat))
    at = int(args[2][0, 32])       # keys 512 .. 527: nodes 16 .. 31 of the first tree
    low = (torch.arange(48, device=gpu) >= 16) & (torch.arange(48, device=gpu) < 32)
    for scales in (cache.k_scales, cache.v_scales):
        for value in (float("nan"), float("inf"), 1e30):
            keep = scales[at].clone()
            scales[at] = value
            got = run()
            torch.cuda.synchronize()
            scales[at] = keep
            if value == 1e30:
                assert torch.equal(got[0][~low], want[~low]) and torch.equal(got[1][~low], wl[~low])
            else:
                others(low, got)


def test_hook_refuses(gpu):
    from post_int4_weight_amd import api
    Q, cache, args, _ = _make(api, gpu, [30], [[-1, 0]], 2, 1, 256, 16, "bf16", 3)
    for plan in ((2, 8, 1), (3, 4, 1), (-1, 4, 1), (0, 2, 1), (1, 4, 1), (0, 8, 1), (1, 8, 1), (0, 4, 0), (0, 4, 65)):
        with pytest.raises(api.PTQError):
            api._test_attention_int8_tree(*plan, Q, cache, *args)


@pytest.mark.parametrize("plan", [(0, 4, 1), (0, 8, 2), (1, 8, 1), (1, 8, 3), (2, 4, 1), (2, 8, 2)])
@pytest.mark.parametrize("batch", [2, 63, 64, 65])
def test_the_order_of_sequences(gpu, batch, plan):
    """Ragged batches of more workgroups than start at once, whose longest sequences go first: equal lengths, sequences
    without rows or keys, one longer than its row of the table."""
    from post_int4_weight_amd import api
    announce(f"tree kernels, order of {batch} sequences, plan {plan}")
    rng = np.random.default_rng(batch)
    prefix = [int(x) for x in rng.integers(0, 30, batch) * rng.integers(0, 30, batch)]
    nodes = [int(x) for x in rng.integers(0, 9, batch)]
    prefix[0], nodes[:2], heads, kv = 800, [5, 40], 32 if batch > 2 else 256, 8 if batch > 2 else 128
    Q, cache, args, vals = _make(api, gpu, prefix, _trees(nodes, 3, batch), heads, kv, 64, 32, "bf16", seed=batch)
    O, lse = api._test_attention_int8_tree(*plan, Q, cache, *args)
    torch.cuda.synchronize()
    _check(O, lse, Q, vals, _trees(nodes, 3, batch), heads, kv, 64 ** -0.5, 0)
    args[1] = args[1].clone()
    args[1][0] = args[2].shape[1] * 32 + 1
    P, _ = api._test_attention_int8_tree(*plan, Q, cache, *args)
    assert torch.isnan(P[:nodes[0]]).all() and torch.equal(P[nodes[0]:], O[nodes[0]:])


@pytest.mark.parametrize("plan,dim", [(p, d) for p in PLANS for d in (64, 128, 256) if _fits(p, d)])
def test_bf16_queries_are_exact(gpu, plan, dim):
    """Rows whose elements are at least 1 / 64 of the largest are held exactly, whatever that one's bits (all 8 set among
    them) and the sign of the softmax scale: lse is off by fp32's roundings alone. A logit C, u = 2^-24: the sums over
    channels round D / 16 + 2 times where they are not exact, the factors and the maximum's subtraction 10 times: (D / 16 +
    12) u (C + 8); the sum of N probabilities (N / 16 + 24) 2 u; and 2 u |lse| for its logarithm's scale, 2^-20 for the
    logarithms."""
    from post_int4_weight_amd import api
    announce(f"tree kernels, exact queries, plan {plan} dim={dim}")
    trees = [[-1, 0, 0, 2], [-1] + [i // 2 for i in range(30)]]
    Q, cache, args, vals = _make(api, gpu, [300, 1000], trees, 4, 2, dim, 32, "bf16", 11)
    gen = torch.Generator().manual_seed(12)
    row = torch.exp2(torch.randint(-20, 4, (Q.shape[0], 4, 1), generator=gen).float())
    size = torch.exp2(-5 * torch.rand(Q.shape, generator=gen)) * row
    Q = (size * (2 * torch.randint(0, 2, Q.shape, generator=gen) - 1)).bfloat16()
    Q[::3, :, 5] = Q[::3].abs().amax(2).float().log2().floor().exp2().mul(255 / 128).bfloat16()      # all bits set
    Q = Q.to(gpu)
    for scale in (dim ** -0.5, -0.05):
        O, lse = api._test_attention_int8_tree(*plan, Q, cache, *args, scale=scale)
        torch.cuda.synchronize()
        q, got, first, u = to64(Q), to64(lse), 0, 2.0 ** -24
        for (k, v), parents in zip(vals, trees):
            base = k.shape[0] - len(parents)
            for i in range(len(parents)):
                keys = ref.keys_of(parents, i, base, 0)
                for h in range(4):
                    _, want, _, _, C = ref.attend(q[first + i, h], k[keys, h // 2], v[keys, h // 2], scale)
                    tol = (dim / 16 + 12) * u * (C + 8) + (len(keys) / 16 + 24) * 2 * u + 2 * u * abs(want) + 2.0 ** -20
                    assert abs(got[first + i, h] - want) <= tol, (i, h, got[first + i, h], want, tol)
            first += len(parents)
