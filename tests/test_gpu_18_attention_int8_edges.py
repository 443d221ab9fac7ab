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
