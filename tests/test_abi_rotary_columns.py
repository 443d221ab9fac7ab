"""rotary_apply's check of where Y lies, without a GPU: columns of Y that reach into X's are refused, also by a row further on."""
import ctypes

import pytest

from post_int4_weight_amd import api

lib = api._lib
BASE = 1 << 20      # never dereferenced: validation fails first


@pytest.mark.parametrize("by", [64, 128 + 64, 512 - 64, 512 + 64, 3 * 512 - 64, -64, -128 - 64, -512 + 64, 512, -512])
def test_columns_that_overlap(by):
    """X: 128 of the 256 columns of 4 rows, bf16; Y the same, `by` bytes further on (rows of 512, X's 256 wide)."""
    status = lib.rotary_apply(ctypes.c_void_p(BASE), 256, ctypes.c_void_p(BASE + by), 256, 0, 4, 2, 64, ctypes.c_void_p(BASE),
                              ctypes.c_void_p(BASE), 32, 0, 1.0, None)
    assert status == 1 and b"overlaps" in lib.ptq_last_error()


@pytest.mark.parametrize("rows,by,ldy", [(4, 256, 264), (1, 64, 256)])
def test_other_strides_and_single_rows(rows, by, ldy):
    status = lib.rotary_apply(ctypes.c_void_p(BASE), 256, ctypes.c_void_p(BASE + by), ldy, 0, rows, 2, 64, ctypes.c_void_p(BASE),
                              ctypes.c_void_p(BASE), 32, 0, 1.0, None)
    assert status == 1 and b"overlaps" in lib.ptq_last_error()
