"""C ABI and Python checks of the drafted-token operators that need no GPU: bad arguments are refused with a message before
any HIP call, empty calls do nothing, tensors on the host never reach the GPU."""
import ctypes

import pytest
import torch

from post_int4_weight_amd import api

lib = api._lib
P = ctypes.c_void_p(1 << 20)           # never dereferenced: validation fails first
FAR = ctypes.c_void_p(1 << 40)
ODD = ctypes.c_void_p((1 << 20) + 4)   # not 16-byte aligned


def _refused(status, word):
    assert status == 1 and word in lib.ptq_last_error().decode(), (status, lib.ptq_last_error())


def test_rotary():
    def call(X=P, ldx=128, Y=FAR, ldy=128, dt=0, rows=4, heads=2, dim=64, pos=P, freq=P, rot=32, il=0, m=1.0):
        return lib.rotary_apply(X, ldx, Y, ldy, dt, rows, heads, dim, pos, freq, rot, il, m, None)
    for word, kw in (("rows", dict(rows=-1)), ("rows", dict(rows=1 << 31)), ("heads", dict(heads=0)),
                     ("head_dim", dict(dim=60)), ("head_dim", dict(dim=0)), ("rotary_dim", dict(rot=66)),
                     ("rotary_dim", dict(rot=31)), ("rotary_dim", dict(rot=0)), ("interleaved", dict(il=2)),
                     ("magnitude", dict(m=float("inf"))), ("dtype", dict(dt=2)), ("X is NULL", dict(X=None)),
                     ("X is not", dict(X=ODD)), ("row stride", dict(ldx=120)), ("row stride", dict(ldy=132)),
                     ("Y is NULL", dict(Y=None)), ("positions", dict(pos=None)), ("inv_freq is NULL", dict(freq=None)),
                     ("inv_freq is not", dict(freq=ODD)), ("overlaps", dict(Y=ctypes.c_void_p((1 << 20) + 256))),
                     ("overlaps", dict(Y=P, ldy=136)), ("too many", dict(rows=(1 << 31) - 1, heads=64, ldx=4096, ldy=4096,
                                                                         Y=ctypes.c_void_p(1 << 60)))):
        _refused(call(**kw), word)
    assert call(rows=0, X=None, Y=None, pos=None, freq=None) == 0


def test_append():
    def call(k=P, nb=10, h=2, d=64, bs=16, K=P, ldk=128, V=P, dt=0, rows=5, off=P, st=P, batch=2, table=P, width=3, pos=None,
             freq=P, rot=64, il=0, m=1.0):
        return lib.kv_cache_append_int8(k, P, P, P, nb, h, d, bs, K, ldk, V, 128, dt, rows, off, st, batch, table, width, pos,
                                        freq, rot, il, m, None)
    for word, kw in (("kv_heads", dict(h=0)), ("head_dim", dict(d=80)), ("block_size", dict(bs=48)), ("negative", dict(rows=-1)),
                     ("rotary_dim", dict(rot=66)), ("rotary_dim", dict(rot=3)), ("interleaved", dict(il=-1)),
                     ("magnitude", dict(m=float("nan"))), ("offsets", dict(off=None)), ("starts", dict(st=None)),
                     ("cache pointer", dict(k=None)), ("K is NULL", dict(K=None)), ("V is not", dict(V=ODD)),
                     ("row stride", dict(ldk=120)), ("dtype", dict(dt=7)), ("inv_freq is NULL", dict(freq=None)),
                     ("too many for a launch", dict(batch=(1 << 24) - 8, h=1, d=256, bs=128, ldk=256, width=1))):
        if word.startswith("too many"):
            _refused(lib.kv_cache_append_int8(P, P, P, P, 10, 1, 256, 128, P, 256, P, 256, 0, 5, P, P, (1 << 24) - 8, P, 1, None,
                                              P, 64, 0, 1.0, None), word)
        else:
            _refused(call(**kw), word)
    assert call(rows=0) == 0 and call(batch=0) == 0


def test_tree():
    def call(Q=P, ldq=256, O=P, ldo=256, dt=0, rows=5, heads=4, off=P, lens=P, par=P, batch=2, table=P, width=300, k=P, nb=10,
             h=2, d=64, bs=16, scale=0.1, window=0, ws=P, wsb=1 << 40):
        return lib.attention_int8_tree(Q, ldq, O, ldo, None, dt, rows, heads, off, lens, par, batch, table, width, k, P, P, P,
                                       nb, h, d, bs, scale, window, ws, wsb, None)
    for word, kw in (("heads", dict(heads=3)), ("heads", dict(heads=0)), ("head_dim", dict(d=32)), ("block_size", dict(bs=256)),
                     ("scale", dict(scale=float("nan"))), ("window", dict(window=-3)), ("seq_lens", dict(lens=None)),
                     ("parents", dict(par=None)), ("cache pointer", dict(k=None)), ("num_blocks", dict(nb=0)),
                     ("Q is not", dict(Q=ODD)), ("row stride", dict(ldo=250)), ("dtype", dict(dt=9)),
                     ("too large", dict(rows=1 << 40)), ("table_width", dict(width=1 << 31))):
        _refused(call(**kw), word)
    need = lib.attention_int8_tree_workspace_bytes(5, 2, 4, 2, 64, 0, 16, 300, 0)
    assert need > 0
    assert call(wsb=need - 1) == 4 and call(ws=None) == 4
    _refused(call(ws=ctypes.c_void_p((1 << 20) + 8)), "workspace is not")
    assert call(rows=0) == 0 and call(batch=0) == 0
    assert lib.attention_int8_tree_workspace_bytes(5, 2, 4, 3, 64, 0, 16, 300, 0) == 0


def test_verify():
    def call(t=P, ldt=100, d=P, ldd=100, dt=1, rows=5, vocab=100, tok=P, par=P, off=P, batch=2, u=P, r=P, path=P, counts=P,
             next=P, ws=P, wsb=1 << 30):
        return lib.verify_drafts(t, ldt, d, ldd, dt, rows, vocab, tok, par, off, batch, u, r, path, counts, next, ws, wsb,
                                 None)
    for word, kw in (("rows", dict(rows=-1)), ("batch", dict(batch=-1)), ("batch", dict(batch=1 << 22)), ("vocab", dict(vocab=0)),
                     ("vocab", dict(vocab=1 << 31)), ("dtype", dict(dt=3)), ("offsets", dict(off=None)),
                     ("counts", dict(counts=None)), ("next", dict(next=None)), ("target is NULL", dict(t=None)),
                     ("target is not", dict(t=ctypes.c_void_p((1 << 20) + 2))), ("row stride", dict(ldt=99)),
                     ("draft is not", dict(d=ctypes.c_void_p((1 << 20) + 1), dt=0)), ("row stride", dict(ldd=99)),
                     ("tokens", dict(tok=None)), ("parents", dict(par=None)), ("NULL", dict(u=None)), ("NULL", dict(r=None)),
                     ("NULL", dict(path=None))):
        _refused(call(**kw), word)
    assert call(batch=0, off=None) == 0
    assert lib.verify_drafts_workspace_bytes(2, 100) == 0 and lib.verify_drafts_workspace_bytes(0, 1 << 20) == 0
    need = lib.verify_drafts_workspace_bytes(2, 1 << 20)
    assert need > 0
    big = dict(vocab=1 << 20, ldt=1 << 20, ldd=1 << 20)
    assert call(**big, wsb=need - 1) == 4 and call(**big, ws=None) == 4
    _refused(call(**big, ws=ctypes.c_void_p((1 << 20) + 8)), "workspace is not")


def test_verify_hook():
    def call(shares, batch=2, wsb=1 << 30):
        return lib.ptq_test_verify_drafts(shares, P, 100, P, 100, 1, 5, 100, P, P, P, batch, P, P, P, P, P, P, wsb, None)
    for shares in (0, 5, -1):
        _refused(call(shares), "shares")
    _refused(call(4, batch=1 << 20), "batch")
    assert call(4, wsb=lib.ptq_test_verify_drafts_workspace_bytes(4, 2) - 1) == 4


def test_tensors_on_the_host_are_refused():
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    refused = lambda name: pytest.raises(ValueError, match=f"{name} must be on the GPU, not on cpu")
    x, rotary = torch.zeros(3, 2, 64), api.Rotary.make(64, device="cpu")
    with refused("X"):
        api.rotary_apply(x, rotary, ints(3))
    with refused("inv_freq"):
        rotary._args()
    cache = api.KVCacheInt8.empty(4, 2, 64, 16, device="cpu")
    with refused("cache.k"):
        api.kv_cache_append_int8(cache, x, x, ints(2), ints(1), ints(1, 1), rotary)
    with refused("cache.k"):
        api.attention_int8_tree(x, cache, ints(2), ints(1), ints(1, 1), ints(3))
    with refused("target"):
        api.verify_drafts(torch.zeros(3, 10), ints(3), ints(3), ints(2), torch.zeros(3), torch.zeros(1))


def test_shapes_are_refused():
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    rotary = api.Rotary.make(64, device="cpu")
    with pytest.raises(ValueError, match="rows, heads"):
        api.rotary_apply(torch.zeros(3, 128), rotary, ints(3))
    with pytest.raises(ValueError, match="must follow each other"):
        api.rotary_apply(torch.zeros(3, 64, 2).transpose(1, 2), rotary, ints(3))
    with pytest.raises(TypeError, match="dtype"):
        api.rotary_apply(torch.zeros(3, 2, 64), rotary, ints(3), Y=torch.zeros(3, 2, 64).bfloat16())
    with pytest.raises(ValueError, match="rows, vocab"):
        api.verify_drafts(torch.zeros(10), ints(3), ints(3), ints(2), torch.zeros(3), torch.zeros(1))
