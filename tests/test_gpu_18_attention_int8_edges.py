"""GPU: attention_int8_cache at the edges of its arguments: windows without an end, values whose scale is infinite, blocks
that a row does not attend to but whose scales are of another size. Each for the kernel of few rows and for tiles."""
import numpy as np
import pytest
import torch

from gpu_util import announce
from test_gpu_14_kv_cache_int8 import _ints, _offsets
from test_gpu_15_attention_int8 import _simple
from test_gpu_16_attention_int8_tiles import _wide

pytestmark = pytest.mark.gpu

KERNELS = {"rows": _simple, "tiles": _wide}


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 62, 2 ** 31])
def test_window_without_end(gpu, window, kernel):
    """A window longer than any key sequence is none, also for rows before the first key."""
    from post_int4_weight_amd import api
    announce(f"attention, window {window} {kernel}")
    lens, qn = [40, 5, 70], (50, 30, 70)
    cache, table, vals, Q, args = KERNELS[kernel](api, gpu, lens, qn, heads=2)
    want, wl = api.attention_int8_cache(Q, cache, *args, return_lse=True)
    got, lse = api.attention_int8_cache(Q, cache, *args, window=window, return_lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and (want[10:50] != 0).any(-1).all()
    assert torch.equal(got, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
def test_infinite_values(gpu, kernel, dim, dtype):
    """An infinite S_v gives NaN, not infinities, to the rows that attend to it; lse, which V has no part in, stays."""
    from post_int4_weight_amd import api
    announce(f"attention, infinite S_v {kernel} {dim} {dtype}")
    lens, qn = [177, 100], (1, 1) if kernel == "rows" else (60, 30)
    cache, table, vals, Q, args = KERNELS[kernel](api, gpu, lens, qn, dtype, dim=dim)
    clean, want = api.attention_int8_cache(Q, cache, *args, return_lse=True)
    for at in (0, 11):                       # positions 0 .. 15; 176 alone
        bad = int(table[0, at])
        keep = cache.v_scales[bad, 1].clone()
        cache.v_scales[bad, 1] = float("inf")
        got, lse = api.attention_int8_cache(Q, cache, *args, return_lse=True)
        torch.cuda.synchronize()
        cache.v_scales[bad, 1] = keep
        seen = torch.zeros(Q.shape[:2], dtype=torch.bool, device=gpu)
        seen[:qn[0], 2:] = (torch.arange(lens[0] - qn[0], lens[0], device=gpu) >= 16 * at)[:, None]
        assert torch.isnan(got[seen]).all() and torch.isfinite(got[~seen]).all()
        assert torch.allclose(lse, want, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("kernel,q", [("rows", 1), ("rows", 30), ("tiles", 30), ("tiles", 90)])
def test_scales_of_blocks_not_attended(gpu, kernel, q, window, dim, dtype):
    """Blocks before a window may hold another sequence's values by now, and blocks past a row are not its own: whatever
    their scale, they do not cost the row bits. Either answer is within half a step of the probabilities (11 or 21 bits) of
    sum w |v| <= the largest |v| of the row's own keys, and of its own rounding."""
    from post_int4_weight_amd import api
    announce(f"attention, large scales of other rows' blocks {kernel} q={q} window={window} {dim} {dtype}")
    n, bs = 250, 16
    cache, table, vals, Q, args = _simple(api, gpu, [n], (q,), dtype, dim=dim, bs=bs)
    run = lambda: api._test_attention_int8_cache(kernel == "tiles", 4, 1, Q, cache, *args, window=window)
    clean, want = run()
    v = np.abs(vals[0][1]).max(-1)           # [keys, kv heads]
    for at in range(n // bs + 1):
        ids = int(table[0, at])
        keep = cache.v_scales[ids].clone()
        cache.v_scales[ids] = 1e35
        got, lse = run()
        torch.cuda.synchronize()
        cache.v_scales[ids] = keep
        for i in range(q):
            p = n - q + i
            lo = max(0, p - window + 1) if window else 0
            if p >= at * bs and lo < at * bs + bs:
                continue                     # attends to it
            bits, out = (11, 8) if dtype == "bf16" else (21, 20)
            top = torch.tensor(v[lo:p + 1].max(0).repeat(2), device=gpu)[:, None]
            err = (got[i].double() - clean[i].double()).abs()
            tol = 2.0 ** (1 - bits) * top + 2.0 ** (1 - out) * clean[i].double().abs()
            assert (err <= tol).all(), (at, i, float((err / tol).max()))
        assert torch.allclose(lse, want, rtol=1e-5, atol=1e-5)
