"""GPU: each kernel of matmul_int8 and attention_int8_cache at sizes where it can go wrong, whichever the estimates would
choose there: the test hooks (include/ptq_testing.h) name the kernel. Bounds as in the tests of the operators."""
import pytest
import torch

from gpu_util import announce
from test_gpu_13_linear_int8 import DTYPES, _check_product, _w
from test_gpu_14_kv_cache_int8 import _ints, _offsets
from test_gpu_15_attention_int8 import _cache, _check

pytestmark = pytest.mark.gpu

SHAPES = [(256, 256), (128, 256), (128, 128), (64, 64), (64, 32), (32, 32)]      # outputs x tokens


def _product(gpu, shape, nsplit, rows, out, n, dtype, bias, pad=0):
    """matmul_int8 by one kernel; pad: columns beyond the operands' rows and Y's."""
    from post_int4_weight_amd import api
    announce(f"matmul_int8 shape={shape} nsplit={nsplit} rows={rows} out={out} in={n} {dtype} bias={bias} pad={pad}")
    gen = torch.Generator().manual_seed(rows + out)
    wide = lambda r: torch.randint(-128, 128, (r, n + 8 * pad), generator=gen, dtype=torch.int8).to(gpu)[:, :n]
    A, (W, sw) = wide(rows), _w(out, n, gpu, out)
    if pad:
        W = wide(out)
    sa = (torch.rand(rows, generator=gen) + 0.1).to(gpu)
    b = torch.randn(out, generator=gen).to(gpu) if bias else None
    big = torch.full((rows + 9, out + pad), 7.0, device=gpu, dtype=DTYPES[dtype])
    Y = big[8:8 + rows, :out] if pad else big[:rows]
    api._test_matmul_int8(shape, nsplit, A, sa, W, sw, bias=b, Y=Y)
    torch.cuda.synchronize()
    _check_product(Y, A, sa, W, sw, b, (shape, nsplit, rows, out, n))
    Y.fill_(7.0)
    assert torch.all(big == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nsplit", [1, 2, 5])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_product_tiles(gpu, shape, nsplit, dtype):
    """More tiles than one along each side, the last ones ragged; whole and ragged depths of fewer stages than a ring, as
    many, and more; rows of Y that are aligned and that are not; fewer rows and outputs than a tile."""
    to, tt = SHAPES[shape]
    bf16 = dtype == "bf16"
    _product(gpu, shape, nsplit, tt + 3, to + 5, 1096, dtype, bias=bf16, pad=3)
    _product(gpu, shape, nsplit, 2 * tt - 1, 2 * to, 640, dtype, bias=not bf16)
    _product(gpu, shape, nsplit, 3 * tt, 3 * to - 16, 2056, dtype, bias=True)
    _product(gpu, shape, nsplit, 5, 9, 1288, dtype, bias=False)
    if nsplit == 1:
        _product(gpu, shape, nsplit, tt + 1, to, 128, dtype, bias=True)
        _product(gpu, shape, nsplit, tt, to + 24, 136, dtype, bias=False, pad=8)


def test_product_streaming(gpu):
    """More than 16 tokens at a time, and depths below one run of the waves."""
    for rows, out, n, pad in ((40, 70, 2056, 0), (17, 33, 72, 1), (100, 16, 8, 0), (33, 250, 120, 5)):
        for dtype in DTYPES:
            _product(gpu, -1, 1, rows, out, n, dtype, bias=rows % 2 == 0, pad=pad)


KERNELS = {"rows": (0, 4, 1), "rows of 8 waves": (0, 8, 1), "rows in 5 splits": (0, 4, 5), "tiles": (1, 4, 1),
           "tiles in 3 splits": (1, 4, 3)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 37, 300])
@pytest.mark.parametrize("kernel", KERNELS)
def test_attention(gpu, kernel, window, dim, dtype):
    """Prompts and a few tokens next to each other, ragged, over keys enough for every split to have some."""
    from post_int4_weight_amd import api
    announce(f"attention kernel={kernel} window={window} dim={dim} {dtype}")
    lens, qn, heads, kv = [700, 900, 40, 5, 2100], [300, 2, 40, 30, 129], 4, 2
    cache, table, vals = _cache(api, lens, kv, dim, 16 if dim == 64 else 64, gpu, 17)
    Q = (1.5 * torch.randn(sum(qn), heads, dim, generator=torch.Generator().manual_seed(18))).to(DTYPES[dtype]).to(gpu)
    args = (_ints(_offsets(qn), gpu), _ints(lens, gpu), _ints(table, gpu))
    O, lse = api._test_attention_int8_cache(*KERNELS[kernel], Q, cache, *args, window=window)
    again, _ = api._test_attention_int8_cache(*KERNELS[kernel], Q, cache, *args, window=window)
    torch.cuda.synchronize()
    assert torch.equal(O, again)
    _check(O, lse, Q, vals, qn, heads, kv, dim, dim ** -0.5, True, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kernel", ["rows", "rows in 5 splits"])
def test_attention_256_channels(gpu, kernel, dtype):
    from post_int4_weight_amd import api
    announce(f"attention kernel={kernel} dim=256 {dtype}")
    lens, qn = [700, 40, 5, 1500], [40, 2, 9, 1]
    cache, table, vals = _cache(api, lens, 2, 256, 32, gpu, 19)
    Q = torch.randn(sum(qn), 4, 256, generator=torch.Generator().manual_seed(20)).to(DTYPES[dtype]).to(gpu)
    O, lse = api._test_attention_int8_cache(*KERNELS[kernel], Q, cache, _ints(_offsets(qn), gpu), _ints(lens, gpu),
                                            _ints(table, gpu), causal=False)
    torch.cuda.synchronize()
    _check(O, lse, Q, vals, qn, 4, 2, 256, 256 ** -0.5, False, 0)
