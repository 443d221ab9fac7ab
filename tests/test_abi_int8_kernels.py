"""Which kernel the int8 serving operators choose (host code, no GPU): every kernel has sizes that reach it, and the sizes
of the tests that mean a kernel do. The test hooks refuse kernels that do not take the sizes."""
import ctypes

import pytest

from post_int4_weight_amd import api

P = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first


@pytest.mark.parametrize("size,shape,split", [((1, 4096, 4096), -1, False), ((300, 512, 72), -1, False),
                                              ((8192, 8192, 8192), 0, False), ((1000, 5003, 28672), 0, True),
                                              ((777, 5003, 4104), 1, False), ((300, 8192, 8192), 1, True),
                                              ((100, 28672, 4096), 2, False), ((100, 8192, 28672), 2, True),
                                              ((100, 8192, 4096), 3, False), ((37, 8192, 28672), 3, True),
                                              ((32, 28672, 264), 4, False), ((37, 1024, 28672), 4, True),
                                              ((200, 1000, 1032), 5, False), ((64, 1024, 8192), 5, True)])
def test_products(size, shape, split):
    got, nsplit = api._test_matmul_int8_plan(*size)
    assert got == shape and (nsplit > 1) == split
    need = api.matmul_int8_workspace_bytes(*size)
    assert need == api._lib.ptq_test_matmul_int8_workspace_bytes(got, nsplit, *size)


def test_attention():
    plan = api._test_attention_int8_plan
    # one short sequence, a long one, and a batch that fills the card without splits
    assert plan(1, 1, 32, 8, 128, 16, 63) == (0, 8, 1)
    assert plan(1, 1, 32, 8, 128, 16, 1000)[:2] == (0, 4) and plan(1, 1, 32, 8, 128, 16, 1000)[2] > 1
    assert plan(64, 64, 64, 8, 128, 64, 251) == (0, 4, 3)
    assert plan(128, 128, 64, 8, 128, 64, 63) == (0, 4, 1)
    # prompts, in one split and in several; 256 channels never take tiles
    assert plan(12189, 4, 32, 8, 128, 64, 79) == (1, 4, 1)
    tiles, _, nsplit = plan(512, 1, 32, 8, 128, 64, 63)
    assert tiles and nsplit > 1
    assert not plan(12189, 4, 32, 8, 256, 64, 79)[0]
    # the sizes of tests/test_gpu_16_attention_int8_tiles.py: ragged, long, non-finite and graph cases are tiles
    for rows, batch, heads, kv in ((449, 9, 4, 2), (1289, 3, 4, 4), (1289, 3, 8, 2), (1289, 3, 3, 1), (1289, 3, 7, 1),
                                   (450, 2, 4, 2), (120, 1, 4, 2), (200, 1, 4, 2), (453, 2, 4, 2)):
        for dim in (64, 128):
            assert plan(rows, batch, heads, kv, dim, 16, 200_000 // 16)[0], (rows, batch, heads, kv, dim)
    # a window shortens the keys: narrow ones at 64 channels take few rows at a time there
    assert not plan(1340, 2, 32, 1, 64, 64, 3125, 37)[0] and plan(1340, 2, 32, 1, 64, 64, 3125, 300)[0]


def test_refusals():
    def product(shape, nsplit, n=256):
        return api._lib.ptq_test_matmul_int8(shape, nsplit, P, n, P, 4, P, n, P, 8, n, None, 0, P, 8, P, 1 << 40, None)
    for bad in (product(6, 1), product(-2, 1), product(-1, 2), product(0, 3), product(0, 0), product(3, 17, 4096),
                product(3, 1, 120)):
        assert bad == 1

    def attention(tiles, waves, nsplit, dim=64):
        return api._lib.ptq_test_attention_int8_cache(tiles, waves, nsplit, P, 4 * dim, P, 4 * dim, None, 0, 5, 4, P, P,
                                                      2, P, 3, P, P, P, P, 10, 2, dim, 16, 0.1, 1, 0, P, 1 << 40, None)
    for bad in (attention(2, 4, 1), attention(1, 4, 1, 256), attention(0, 8, 1, 256), attention(0, 8, 2),
                attention(1, 8, 1), attention(0, 5, 1), attention(0, 4, 0), attention(0, 4, 65)):
        assert bad == 1
