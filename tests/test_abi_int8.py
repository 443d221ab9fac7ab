"""C ABI checks of the int8 serving operators that need no GPU: bad arguments
are refused with a message before any HIP call, empty calls do nothing."""
import ctypes

import pytest

P = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 4)  # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    from post_int4_weight_amd import api
    return api._lib


def _refused(lib, status, word):
    assert status == 1
    assert word in lib.ptq_last_error().decode()


def test_quantize_tokens(lib):
    def call(X=P, dt=0, rows=4, n=64, ldx=64, s=None, codes=P, ldc=64, scales=P):
        return lib.quantize_tokens_int8(X, dt, rows, n, ldx, s, codes, ldc, scales, None)
    _refused(lib, call(n=60), "multiple of 8")
    _refused(lib, call(n=0), "in = 0")
    _refused(lib, call(n=131072, ldx=131072, ldc=131072), "131064")
    _refused(lib, call(rows=-1), "rows")
    _refused(lib, call(rows=1 << 31), "rows")
    _refused(lib, call(dt=2), "dtype")
    _refused(lib, call(X=None), "X is NULL")
    _refused(lib, call(X=ODD), "aligned")
    _refused(lib, call(ldx=68), "row stride")
    _refused(lib, call(ldx=56), "row stride")
    _refused(lib, call(s=ODD), "s is not")
    _refused(lib, call(codes=None), "codes is NULL")
    _refused(lib, call(ldc=63), "row stride")
    _refused(lib, call(scales=None), "scales is NULL")
    assert call(rows=0, X=None, codes=None, scales=None) == 0


def test_matmul(lib):
    def call(A=P, lda=64, sa=P, rows=4, B=P, ldb=64, sb=P, out=8, n=64, dt=0, Y=P, ldy=8, ws=P, wsb=1 << 40):
        return lib.matmul_int8(A, lda, sa, rows, B, ldb, sb, out, n, None, dt, Y, ldy, ws, wsb, None)
    _refused(lib, call(n=4), "multiple of 8")
    _refused(lib, call(out=-1), "out")
    _refused(lib, call(rows=(1 << 31) - 1, out=(1 << 31) - 1), "too large")
    _refused(lib, call(A=None), "A is NULL")
    _refused(lib, call(A=ODD), "A is not")
    _refused(lib, call(lda=60), "row stride")
    _refused(lib, call(sa=None), "a_scales")
    _refused(lib, call(B=None), "codes is NULL")
    _refused(lib, call(ldb=68), "row stride")
    _refused(lib, call(sb=None), "scales is NULL")
    _refused(lib, call(dt=5), "dtype of Y")
    _refused(lib, call(Y=None), "Y is NULL")
    _refused(lib, call(ldy=7), "row stride")
    assert call(rows=0) == 0 and call(out=0) == 0
    assert lib.matmul_int8_workspace_bytes(0, 8, 64) == 0


def test_linear(lib):
    need = lib.linear_int8_workspace_bytes(4, 8, 64)
    assert need >= 4 * 64 + 16

    def call(X=P, dt=0, rows=4, ldx=64, s=None, B=P, ldb=64, sb=P, out=8, n=64, ydt=0, Y=P, ldy=8, ws=P, wsb=need):
        return lib.linear_int8(X, dt, rows, ldx, s, B, ldb, sb, out, n, None, ydt, Y, ldy, ws, wsb, None)
    _refused(lib, call(n=63), "multiple of 8")
    _refused(lib, call(dt=7), "dtype of X")
    _refused(lib, call(X=ODD), "X is not")
    _refused(lib, call(ldx=60), "row stride")
    _refused(lib, call(s=ODD), "s is not")
    _refused(lib, call(B=ODD), "codes is not")
    _refused(lib, call(ydt=3), "dtype of Y")
    _refused(lib, call(Y=ODD), "Y is not")
    _refused(lib, call(ws=ctypes.c_void_p((1 << 20) + 8)), "workspace is not")
    assert call(ws=None) == 4 and call(wsb=need - 1) == 4
    assert "need" in lib.ptq_last_error().decode()
    assert call(rows=0) == 0


@pytest.mark.parametrize("name", ["kv_cache_write_int8", "kv_cache_read_int8"])
def test_cache(lib, name):
    def call(k=P, v=P, ks=P, vs=P, nb=10, h=2, d=64, bs=16, K=P, ldk=128, V=P, ldv=128, dt=0, rows=5, off=P, st=P,
             batch=2, table=P, width=3):
        return getattr(lib, name)(k, v, ks, vs, nb, h, d, bs, K, ldk, V, ldv, dt, rows, off, st, batch, table, width,
                                  None)
    _refused(lib, call(h=0), "kv_heads")
    _refused(lib, call(d=80), "head_dim")
    _refused(lib, call(bs=8), "block_size")
    _refused(lib, call(bs=48), "block_size")
    _refused(lib, call(nb=-1), "num_blocks")
    _refused(lib, call(rows=-1), "negative")
    _refused(lib, call(batch=-1), "negative")
    _refused(lib, call(rows=1 << 40), "too large")
    _refused(lib, call(width=1 << 31), "table_width")
    _refused(lib, call(off=None), "offsets")
    _refused(lib, call(st=None), "starts")
    _refused(lib, call(table=None), "block_table")
    _refused(lib, call(k=None), "cache pointer")
    _refused(lib, call(vs=None), "cache pointer")
    _refused(lib, call(v=ODD), "aligned")
    _refused(lib, call(K=None), "K is NULL")
    _refused(lib, call(V=ODD), "V is not")
    _refused(lib, call(ldk=120), "row stride")
    _refused(lib, call(ldv=132), "row stride")
    _refused(lib, call(dt=-1), "dtype")
    assert call(rows=0) == 0 and call(batch=0) == 0


def test_attention(lib):
    def call(Q=P, ldq=256, O=P, ldo=256, dt=0, rows=5, heads=4, off=P, lens=P, batch=2, table=P, width=300, k=P, nb=10,
             h=2, d=64, bs=16, scale=0.1, causal=1, window=0, ws=P, wsb=1 << 40):
        return lib.attention_int8_cache(Q, ldq, O, ldo, None, dt, rows, heads, off, lens, batch, table, width, k, P, P,
                                        P, nb, h, d, bs, scale, causal, window, ws, wsb, None)
    _refused(lib, call(heads=3), "heads")
    _refused(lib, call(heads=0), "heads")
    _refused(lib, call(d=32), "head_dim")
    _refused(lib, call(bs=256), "block_size")
    _refused(lib, call(scale=float("nan")), "scale")
    _refused(lib, call(causal=2), "causal")
    _refused(lib, call(window=-3), "window")
    _refused(lib, call(causal=0, window=3), "window")
    _refused(lib, call(lens=None), "seq_lens")
    _refused(lib, call(k=None), "cache pointer")
    _refused(lib, call(nb=0), "num_blocks")
    _refused(lib, call(Q=ODD), "Q is not")
    _refused(lib, call(ldo=250), "row stride")
    _refused(lib, call(dt=9), "dtype")
    need = lib.attention_int8_cache_workspace_bytes(5, 2, 4, 2, 64, 16, 300)
    assert need > 0
    assert call(wsb=need - 1) == 4 and call(ws=None) == 4
    _refused(lib, call(ws=ctypes.c_void_p((1 << 20) + 8)), "workspace is not")
    assert call(rows=0) == 0
    assert lib.attention_int8_cache_workspace_bytes(5, 2, 4, 3, 64, 16, 300) == 0
