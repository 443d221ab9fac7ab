"""Refusals of the int8 serving operators in the C ABI that need no GPU: workspaces that are not aligned, sizes past what a
launch takes."""
import ctypes

from post_int4_weight_amd import api

lib = api._lib
P = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned


def _refused(status, word):
    assert status == 1 and word in lib.ptq_last_error().decode()


def test_matmul_workspace_alignment():
    """Partial sums and staged codes are read and written 16 bytes at a time, and copied into LDS."""
    for rows, out, n in ((40, 200, 264), (300, 8192, 8192), (777, 5003, 4104)):     # ragged depth, split depth, both
        need = lib.matmul_int8_workspace_bytes(rows, out, n)
        assert need > 0
        _refused(lib.matmul_int8(P, n, P, rows, P, n, P, out, n, None, 0, P, out, ODD, need, None), "workspace is not")


def test_launches_of_2_32_threads():
    """Sequences are looked up in the launch, which has workgroups for each: as many as wrap its size are refused."""
    for name in ("kv_cache_write_int8", "kv_cache_read_int8"):
        for dtype in (0, 1):
            _refused(getattr(lib, name)(P, P, P, P, 10, 1, 256, 128, P, 256, P, 256, dtype, 5, P, P, (1 << 24) - 8, P, 1,
                                        None), "too many for a launch")
