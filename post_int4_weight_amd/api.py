"""ctypes binding of libptq.so — argument marshalling only.

Every function takes torch tensors that already live on the GPU, passes their
device pointers, sizes and torch's current HIP stream to the C entry point of
the same name (include/ptq.h), and raises PTQError on a non-OK status. Output
tensors may be passed in (no allocation) or are allocated here with
torch.empty; workspaces likewise. Nothing here computes: there is no CPU or
PyTorch fallback, and a missing library is an ImportError.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

PTQ_BF16 = 0
PTQ_F32 = 1

_STATUS = {0: "PTQ_OK", 1: "PTQ_EINVAL", 2: "PTQ_ENOTPD", 3: "PTQ_ENONFINITE", 4: "PTQ_EWORKSPACE",
           5: "PTQ_EHIP"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libptq.so")


class PTQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status
        self.name = _STATUS.get(status, str(status))


def library_path() -> str:
    return _LIB_PATH


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with `python post_int4_weight_amd/build.py`")
    lib = ctypes.CDLL(_LIB_PATH)
    i64, i32, sz, vp, dbl = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_double
    fp = ctypes.POINTER(ctypes.c_float)
    dp = ctypes.POINTER(ctypes.c_double)
    sig = {
        "ptq_last_error": (ctypes.c_char_p, []),
        "ptq_status_string": (ctypes.c_char_p, [i32]),
        "ptq_abi_version": (i32, []),
        "ptq_profile_enable": (i32, [ctypes.c_uint]),
        "ptq_profile_read": (i32, [i32, dp, ctypes.POINTER(i64)]),
        "ptq_profile_flops": (i32, [i32, dp]),
        "hessian_workspace_bytes": (sz, [i64, i64]),
        "hessian_accumulate": (i32, [vp, vp, i64, vp, i32, i64, i64, vp, sz, vp]),
        "hessian_accumulate_noalloc": (i32, [vp, vp, i64, vp, i32, i64, i64, vp]),
        "gptq_factor_workspace_bytes": (sz, [i64]),
        "gptq_inverse_factor": (i32, [vp, vp, i64, dbl, i32, vp, vp, dp, vp, sz, vp]),
        "gptq_columns_workspace_bytes": (sz, [i64, i64, i32]),
        "gptq_quantize_columns": (i32, [vp, i32, i64, i64, i64, vp, vp, i32, i32, i32, vp, vp, vp, dp, vp, sz, vp]),
        "gptq_workspace_bytes": (sz, [i64, i64, i32]),
        "gptq_quantize_layer": (i32, [vp, i32, i64, i64, i64, vp, vp, i32, i32, dbl, i32, i32, vp, vp, vp, vp, dp,
                                      vp, sz, vp]),
        "awq_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "ptq_test_gemm_f32": (i32, [i64, i64, i64, vp, i64, i32, vp, i64, i32, vp, i64, ctypes.c_float, i32, i32,
                                    i32, vp]),
        "awq_search_alpha": (i32, [vp, i32, i64, i64, i64, vp, i32, i64, i64, fp, i32, i32, i32, fp, dp, vp, vp, vp,
                                   vp, sz, vp]),
        "pack_int4": (i32, [vp, i64, i64, i32, vp, vp]),
        "awq_gptq_quantize_layer_workspace_bytes": (sz, [i64, i64, i32]),
        "awq_gptq_quantize_layer": (i32, [vp, i32, i64, i64, i64, vp, vp, vp, i32, i32, dbl, i32, i32, vp, vp, vp, vp,
                                          dp, vp, sz, vp]),
        "dequantize_int4": (i32, [vp, vp, vp, vp, i64, i64, i32, i32, vp, i64, vp]),
        "gptq_quantize_layer_zp": (i32, [vp, i32, i64, i64, i64, vp, vp, i32, i32, dbl, i32, i32, vp, vp, vp, vp, vp,
                                         dp, vp, sz, vp]),
        "layer_output_error_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "ptq_test_gemm_f32_pair": (i32, [i64, i64, i64, vp, i64, vp, i64, vp, i64, ctypes.c_float, i32, i32, i32,
                                         i64, i64, i64, vp, i64, vp, i64, vp, i64, ctypes.c_float, i32, i32, i32,
                                         vp]),
        "ptq_test_gemm_f32_split3_workspace_bytes": (sz, [i64, i64, i64]),
        "ptq_test_gemm_f32_split3": (i32, [i64, i64, i64, vp, i64, i32, vp, i64, i32, vp, i64, ctypes.c_float, i32,
                                           i32, i32, vp, sz, vp]),
        "quantize_tokens_int8": (i32, [vp, i32, i64, i64, i64, vp, vp, i64, vp, vp]),
        "matmul_int8_workspace_bytes": (sz, [i64, i64, i64]),
        "matmul_int8": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, i32, vp, i64, vp, sz, vp]),
        "linear_int8_workspace_bytes": (sz, [i64, i64, i64]),
        "linear_int8": (i32, [vp, i32, i64, i64, vp, vp, i64, vp, i64, i64, vp, i32, vp, i64, vp, sz, vp]),
        "kv_cache_write_int8": (i32, [vp, vp, vp, vp, i64, i32, i32, i32, vp, i64, vp, i64, i32, i64, vp, vp, i64,
                                      vp, i64, vp]),
        "kv_cache_read_int8": (i32, [vp, vp, vp, vp, i64, i32, i32, i32, vp, i64, vp, i64, i32, i64, vp, vp, i64,
                                     vp, i64, vp]),
        "attention_int8_cache_workspace_bytes": (sz, [i64, i64, i32, i32, i32, i32, i64]),
        "attention_int8_cache": (i32, [vp, i64, vp, i64, vp, i32, i64, i32, vp, vp, i64, vp, i64, vp, vp, vp, vp,
                                       i64, i32, i32, i32, ctypes.c_float, i32, i64, vp, sz, vp]),
        "ptq_test_matmul_int8_plan": (i32, [i64, i64, i64, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "ptq_test_matmul_int8_workspace_bytes": (sz, [i32, i32, i64, i64, i64]),
        "ptq_test_matmul_int8": (i32, [i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, i32, vp, i64, vp, sz,
                                       vp]),
        "ptq_test_attention_int8_plan": (i32, [i64, i64, i32, i32, i32, i32, i64, i64, ctypes.POINTER(i32),
                                               ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "ptq_test_attention_int8_workspace_bytes": (sz, [i32, i64, i32, i32]),
        "ptq_test_attention_int8_cache": (i32, [i32, i32, i32, vp, i64, vp, i64, vp, i32, i64, i32, vp, vp, i64, vp,
                                                i64, vp, vp, vp, vp, i64, i32, i32, i32, ctypes.c_float, i32, i64,
                                                vp, sz, vp]),
        "layer_output_error": (i32, [vp, i32, i64, i64, vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, i32, dp, vp, sz,
                                     vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def _check(status: int):
    if status != 0:
        raise PTQError(status, _lib.ptq_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    # torch.cuda.current_stream().cuda_stream without the Stream object (0.3 us instead of 2.8)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PTQ_BF16
    if t.dtype == torch.float32:
        return PTQ_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _workspace(nbytes: int, device, given):
    if given is not None:
        return given, given.numel() * given.element_size()
    if nbytes == 0:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def _rowmajor(t: torch.Tensor, name: str):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D row-major tensor")
    return t.stride(0)


# ------------------------------------------------------------- profiling ---

PROFILE_KERNELS = {"xtx_gemm": 0, "factor_gemm": 1, "factor_base": 2, "block_loop": 3, "trail_gemm": 4,
                   "awq_gemm": 5, "inner_gemm": 6, "split3_gemm": 7}


def profile_enable(kernels=()):
    """Bracket later launches of the named kernel classes with hipEvents."""
    mask = 0
    for k in kernels:
        mask |= 1 << PROFILE_KERNELS[k]
    _check(_lib.ptq_profile_enable(mask))


def profile_read(kernel: str):
    """(total_ms, launches) of the recorded launches of one kernel class."""
    tot = ctypes.c_double(0.0)
    cnt = ctypes.c_int64(0)
    _check(_lib.ptq_profile_read(PROFILE_KERNELS[kernel], ctypes.byref(tot), ctypes.byref(cnt)))
    return tot.value, cnt.value


def profile_flops(kernel: str) -> float:
    """MFMA flops executed by the recorded launches of one kernel class."""
    f = ctypes.c_double(0.0)
    _check(_lib.ptq_profile_flops(PROFILE_KERNELS[kernel], ctypes.byref(f)))
    return f.value


# ---------------------------------------------------------------- stage 1 ---

def hessian_workspace_bytes(n: int, rows: int) -> int:
    return int(_lib.hessian_workspace_bytes(n, rows))


def hessian_accumulate(H: torch.Tensor, d: torch.Tensor | None, X: torch.Tensor, workspace=None):
    """H (+)= X^T X (fp32 [n, n]), d (+)= column sums of squares (fp64 [n])."""
    n = H.shape[0]
    ldx = _rowmajor(X, "X")
    ws, wsb = _workspace(hessian_workspace_bytes(n, X.shape[0]), X.device, workspace)
    _check(_lib.hessian_accumulate(_ptr(H), _ptr(d), n, _ptr(X), _dtype_code(X), X.shape[0], ldx, _ptr(ws), wsb,
                                   _stream()))
    return H, d


def hessian_accumulate_noalloc(H: torch.Tensor, d: torch.Tensor | None, X: torch.Tensor):
    """hessian_accumulate_noalloc (include/ptq.h): the same sums with the
    library's fixed device scratch instead of a workspace (allocates nothing)."""
    n = H.shape[0]
    ldx = _rowmajor(X, "X")
    _check(_lib.hessian_accumulate_noalloc(_ptr(H), _ptr(d), n, _ptr(X), _dtype_code(X), X.shape[0], ldx,
                                           _stream()))
    return H, d


# ---------------------------------------------------------------- stage 2 ---

def gptq_factor_workspace_bytes(n: int) -> int:
    return int(_lib.gptq_factor_workspace_bytes(n))


def gptq_inverse_factor(H, d=None, damp=0.01, act_order=False, U=None, perm=None, workspace=None):
    """Upper factor U of (P (H + lambda I) P^T)^-1; returns (U, perm, lambda)."""
    n = H.shape[0]
    if U is None:
        U = torch.empty(n, n, dtype=torch.float32, device=H.device)
    if perm is None and act_order:
        perm = torch.empty(n, dtype=torch.int32, device=H.device)
    ws, wsb = _workspace(gptq_factor_workspace_bytes(n), H.device, workspace)
    lam = ctypes.c_double(0.0)
    _check(_lib.gptq_inverse_factor(_ptr(H), _ptr(d), n, float(damp), int(bool(act_order)), _ptr(U), _ptr(perm),
                                    ctypes.byref(lam), _ptr(ws), wsb, _stream()))
    return U, perm, lam.value


# ---------------------------------------------------------------- stage 3 ---

def gptq_columns_workspace_bytes(out: int, n: int, block_size: int = 128) -> int:
    return int(_lib.gptq_columns_workspace_bytes(out, n, block_size))


def _alloc_codes(W, n, g, codes, scales, g_idx):
    out = W.shape[0]
    dev = W.device
    if codes is None:
        codes = torch.empty(out, n, dtype=torch.int8, device=dev)
    if scales is None:
        scales = torch.empty(out, (n + g - 1) // g, dtype=torch.float32, device=dev)
    if g_idx is None:
        g_idx = torch.empty(n, dtype=torch.int32, device=dev)
    return codes, scales, g_idx


def gptq_quantize_columns(W, U, perm=None, bits=4, group_size=128, block_size=128, codes=None, scales=None,
                          g_idx=None, workspace=None):
    """The column loop given U; returns (codes, scales, g_idx, stats[4])."""
    out, n = W.shape
    ldw = _rowmajor(W, "W")
    codes, scales, g_idx = _alloc_codes(W, n, group_size, codes, scales, g_idx)
    ws, wsb = _workspace(gptq_columns_workspace_bytes(out, n, block_size), W.device, workspace)
    stats = (ctypes.c_double * 4)()
    _check(_lib.gptq_quantize_columns(_ptr(W), _dtype_code(W), out, n, ldw, _ptr(U), _ptr(perm), bits, group_size,
                                      block_size, _ptr(codes), _ptr(scales), _ptr(g_idx), stats, _ptr(ws), wsb,
                                      _stream()))
    return codes, scales, g_idx, list(stats)


# ------------------------------------------------------------ stages 2+3 ---

def gptq_workspace_bytes(out: int, n: int, block_size: int = 128) -> int:
    return int(_lib.gptq_workspace_bytes(out, n, block_size))


def gptq_quantize_layer(W, H, d=None, bits=4, group_size=128, damp=0.01, act_order=False, block_size=128,
                        codes=None, scales=None, g_idx=None, perm=None, workspace=None):
    """Whole GPTQ layer from the undamped H; returns dict(codes, scales, g_idx, perm, stats)."""
    out, n = W.shape
    ldw = _rowmajor(W, "W")
    codes, scales, g_idx = _alloc_codes(W, n, group_size, codes, scales, g_idx)
    if perm is None:
        perm = torch.empty(n, dtype=torch.int32, device=W.device)
    ws, wsb = _workspace(gptq_workspace_bytes(out, n, block_size), W.device, workspace)
    stats = (ctypes.c_double * 4)()
    _check(_lib.gptq_quantize_layer(_ptr(W), _dtype_code(W), out, n, ldw, _ptr(H), _ptr(d), bits, group_size,
                                    float(damp), int(bool(act_order)), block_size, _ptr(codes), _ptr(scales),
                                    _ptr(g_idx), _ptr(perm), stats, _ptr(ws), wsb, _stream()))
    return {"codes": codes, "scales": scales, "g_idx": g_idx, "perm": perm,
            "stats": {"sum_err2": stats[0], "lambda": stats[1], "dW_fro2": stats[2], "objective": stats[3]}}


# ---------------------------------------------------------------- stage 4 ---

def awq_workspace_bytes(out: int, n: int, rows: int, n_alpha: int) -> int:
    return int(_lib.awq_workspace_bytes(out, n, rows, n_alpha))


def awq_search_alpha(W, X, alphas, bits=4, group_size=128, s=None, codes=None, scales=None, workspace=None):
    """AWQ grid search; returns dict(alpha, errors, s, codes, scales)."""
    out, n = W.shape
    rows = X.shape[0]
    ldw = _rowmajor(W, "W")
    ldx = _rowmajor(X, "X")
    na = len(alphas)
    al = (ctypes.c_float * na)(*[float(a) for a in alphas])
    dev = W.device
    if s is None:
        s = torch.empty(n, dtype=torch.float32, device=dev)
    if codes is None:
        codes = torch.empty(out, n, dtype=torch.int8, device=dev)
    if scales is None:
        scales = torch.empty(out, (n + group_size - 1) // group_size, dtype=torch.float32, device=dev)
    ws, wsb = _workspace(awq_workspace_bytes(out, n, rows, na), dev, workspace)
    best = ctypes.c_float(0.0)
    errs = (ctypes.c_double * na)()
    _check(_lib.awq_search_alpha(_ptr(W), _dtype_code(W), out, n, ldw, _ptr(X), _dtype_code(X), rows, ldx, al, na,
                                 bits, group_size, ctypes.byref(best), errs, _ptr(s), _ptr(codes), _ptr(scales),
                                 _ptr(ws), wsb, _stream()))
    return {"alpha": best.value, "errors": list(errs), "s": s, "codes": codes, "scales": scales}


# ------------------------------------------- composition and INT4 storage ---

def gptq_quantize_layer_zp(W, H, d=None, bits=4, group_size=128, damp=0.01, act_order=False, block_size=128,
                           codes=None, scales=None, zeros=None, g_idx=None, perm=None, workspace=None):
    """gptq_quantize_layer_zp (include/ptq.h): GPTQ with zero-point groups; codes in [0, 2^bits - 1]."""
    out, n = W.shape
    ldw = _rowmajor(W, "W")
    codes, scales, g_idx = _alloc_codes(W, n, group_size, codes, scales, g_idx)
    if zeros is None:
        zeros = torch.empty(out, (n + group_size - 1) // group_size, dtype=torch.int8, device=W.device)
    if perm is None:
        perm = torch.empty(n, dtype=torch.int32, device=W.device)
    ws, wsb = _workspace(gptq_workspace_bytes(out, n, block_size), W.device, workspace)
    stats = (ctypes.c_double * 4)()
    _check(_lib.gptq_quantize_layer_zp(_ptr(W), _dtype_code(W), out, n, ldw, _ptr(H), _ptr(d), bits, group_size,
                                       float(damp), int(bool(act_order)), block_size, _ptr(codes), _ptr(scales),
                                       _ptr(zeros), _ptr(g_idx), _ptr(perm), stats, _ptr(ws), wsb, _stream()))
    return {"codes": codes, "scales": scales, "zeros": zeros, "g_idx": g_idx, "perm": perm,
            "stats": {"sum_err2": stats[0], "lambda": stats[1], "dW_fro2": stats[2], "objective": stats[3]}}


def awq_gptq_quantize_layer(W, H, d, s, bits=4, group_size=128, damp=0.01, act_order=False, block_size=128,
                            codes=None, scales=None, g_idx=None, perm=None, workspace=None):
    """awq_gptq_quantize_layer (include/ptq.h): GPTQ on W diag(s) with the Hessian of X diag(s)^-1."""
    out, n = W.shape
    ldw = _rowmajor(W, "W")
    codes, scales, g_idx = _alloc_codes(W, n, group_size, codes, scales, g_idx)
    if perm is None:
        perm = torch.empty(n, dtype=torch.int32, device=W.device)
    ws, wsb = _workspace(int(_lib.awq_gptq_quantize_layer_workspace_bytes(out, n, block_size)), W.device, workspace)
    stats = (ctypes.c_double * 4)()
    _check(_lib.awq_gptq_quantize_layer(_ptr(W), _dtype_code(W), out, n, ldw, _ptr(H), _ptr(d), _ptr(s), bits,
                                        group_size, float(damp), int(bool(act_order)), block_size, _ptr(codes),
                                        _ptr(scales), _ptr(g_idx), _ptr(perm), stats, _ptr(ws), wsb, _stream()))
    return {"codes": codes, "scales": scales, "g_idx": g_idx, "perm": perm,
            "stats": {"sum_err2": stats[0], "lambda": stats[1], "dW_fro2": stats[2], "objective": stats[3]}}


def pack_int4(codes: torch.Tensor, bits: int = 4, packed=None):
    """pack_int4 (include/ptq.h): int8 codes [out, in] -> int32 words [out, in/8]
    (uint32 bit patterns; torch has no uint32 arithmetic, so int32 holds them)."""
    out, n = codes.shape
    if codes.dtype != torch.int8 or codes.stride(1) != 1 or codes.stride(0) != n:
        raise ValueError("codes must be a contiguous int8 [out, in] tensor")
    if packed is None:
        packed = torch.empty(out, n // 8, dtype=torch.int32, device=codes.device)
    _check(_lib.pack_int4(_ptr(codes), out, n, bits, _ptr(packed), _stream()))
    return packed


def dequantize_int4(packed: torch.Tensor, scales: torch.Tensor, g_idx, n: int, group_size: int = 128,
                    out_dtype=torch.float32, What=None, zeros=None):
    """dequantize_int4 (include/ptq.h): What[r][c] = code * scales[r][g_idx[c]] (g_idx None: c // group_size);
    with zeros, unsigned codes and What = (code - zero) * scale."""
    out = packed.shape[0]
    if What is None:
        What = torch.empty(out, n, dtype=out_dtype, device=packed.device)
    ldo = _rowmajor(What, "What") if out > 0 else n
    _check(_lib.dequantize_int4(_ptr(packed), _ptr(scales), _ptr(g_idx), _ptr(zeros), out, n, group_size,
                                _dtype_code(What), _ptr(What), ldo, _stream()))
    return What


# ------------------------------------------------------------ evaluation ---

def layer_output_error_workspace_bytes(out: int, n: int, rows: int, x_dtype: int) -> int:
    return int(_lib.layer_output_error_workspace_bytes(out, n, rows, x_dtype))


def layer_output_error(X, W, codes, scales, g_idx=None, zeros=None, s=None, group_size=128, workspace=None):
    """layer_output_error (include/ptq.h): (||X (W - What)^T||^2, ||X W^T||^2) with
    What = (codes - zeros[g_idx]) * scales[g_idx] / s."""
    out, n = W.shape
    rows = X.shape[0]
    ldw = _rowmajor(W, "W")
    ldx = _rowmajor(X, "X")
    if codes.dtype != torch.int8 or not codes.is_contiguous() or tuple(codes.shape) != (out, n):
        raise ValueError("codes must be a contiguous int8 [out, in] tensor")
    xd = _dtype_code(X)
    ws, wsb = _workspace(layer_output_error_workspace_bytes(out, n, rows, xd), W.device, workspace)
    res = (ctypes.c_double * 2)()
    _check(_lib.layer_output_error(_ptr(X), xd, rows, ldx, _ptr(W), _dtype_code(W), out, n, ldw, _ptr(codes),
                                   _ptr(scales), _ptr(g_idx), _ptr(zeros), _ptr(s), group_size, res, _ptr(ws), wsb,
                                   _stream()))
    return res[0], res[1]


# ---------------------------------------------------------- int8 serving ---

def _on_gpu(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, not on {t.device}")


def _vector(t, n: int, dtype, name: str):
    """t as n dense values of dtype (any shape with that many), or None."""
    if t is None:
        return None
    _on_gpu(t, name)
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous {dtype} values")
    return t.data_ptr()


def _codes(t: torch.Tensor, name: str):
    if t.dtype != torch.int8:
        raise TypeError(f"{name} must be int8, not {t.dtype}")
    return _rows(t, name)


def _rows(t: torch.Tensor, name: str):
    ld = _rowmajor(t, name)
    _on_gpu(t, name)
    return ld


def _scratch(nbytes: int, device, given):
    if given is not None:
        _on_gpu(given, "workspace")
    return _workspace(nbytes, device, given)


def quantize_tokens_int8(X: torch.Tensor, s=None, codes=None, scales=None):
    """quantize_tokens_int8 (include/ptq.h): X [rows, in] -> (codes int8 [rows, in], scales fp32 [rows]); s divides
    the columns first."""
    rows, n = X.shape
    ldx = _rows(X, "X")
    if codes is None:
        codes = torch.empty(rows, n, dtype=torch.int8, device=X.device)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=X.device)
    if tuple(codes.shape) != (rows, n):
        raise ValueError("codes must be [rows, in]")
    _check(_lib.quantize_tokens_int8(_ptr(X), _dtype_code(X), rows, n, ldx, _vector(s, n, torch.float32, "s"),
                                     _ptr(codes), _codes(codes, "codes"),
                                     _vector(scales, rows, torch.float32, "scales"), _stream()))
    return codes, scales


def matmul_int8_workspace_bytes(rows: int, out: int, n: int) -> int:
    return int(_lib.matmul_int8_workspace_bytes(rows, out, n))


def _product_output(Y, rows, out, dtype, device):
    if Y is None:
        return torch.empty(rows, out, dtype=dtype, device=device), max(out, 1)
    if tuple(Y.shape) != (rows, out):
        raise ValueError("Y must be [rows, out]")
    ldy = _rows(Y, "Y")
    return Y, ldy if rows > 1 else max(out, 1)


def matmul_int8(A, a_scales, codes, scales, bias=None, out_dtype=torch.bfloat16, Y=None, workspace=None):
    """matmul_int8 (include/ptq.h): Y[t][o] = (A codes^T)[t][o] * a_scales[t] * scales[o] + bias[o]."""
    rows, n = A.shape
    out = codes.shape[0]
    if codes.shape[1] != n:
        raise ValueError(f"codes has {codes.shape[1]} columns, A has {n}")
    Y, ldy = _product_output(Y, rows, out, out_dtype, A.device)
    ws, wsb = _scratch(matmul_int8_workspace_bytes(rows, out, n), A.device, workspace)
    _check(_lib.matmul_int8(_ptr(A), _codes(A, "A"), _vector(a_scales, rows, torch.float32, "a_scales"), rows,
                            _ptr(codes), _codes(codes, "codes"), _vector(scales, out, torch.float32, "scales"), out, n,
                            _vector(bias, out, torch.float32, "bias"), _dtype_code(Y), _ptr(Y), ldy, _ptr(ws), wsb,
                            _stream()))
    return Y


def linear_int8_workspace_bytes(rows: int, out: int, n: int) -> int:
    return int(_lib.linear_int8_workspace_bytes(rows, out, n))


def linear_int8(X, codes, scales, bias=None, s=None, out_dtype=None, Y=None, workspace=None):
    """linear_int8 (include/ptq.h): X [rows, in] through int8 codes [out, in] with one scale per output channel
    (group_size = in of the quantizers); the activations are quantized token by token. Y has X's dtype unless
    out_dtype says otherwise."""
    rows, n = X.shape
    out = codes.shape[0]
    if codes.shape[1] != n:
        raise ValueError(f"codes has {codes.shape[1]} columns, X has {n}")
    Y, ldy = _product_output(Y, rows, out, out_dtype or X.dtype, X.device)
    ws, wsb = _scratch(linear_int8_workspace_bytes(rows, out, n), X.device, workspace)
    _check(_lib.linear_int8(_ptr(X), _dtype_code(X), rows, _rows(X, "X"), _vector(s, n, torch.float32, "s"),
                            _ptr(codes), _codes(codes, "codes"), _vector(scales, out, torch.float32, "scales"), out, n,
                            _vector(bias, out, torch.float32, "bias"), _dtype_code(Y), _ptr(Y), ldy, _ptr(ws), wsb,
                            _stream()))
    return Y


class KVCacheInt8(NamedTuple):
    """The four tensors of an int8 key/value cache (layout in include/ptq.h)."""
    k: torch.Tensor           # int8 [num_blocks, kv_heads, block_size, head_dim]
    v: torch.Tensor           # int8 [num_blocks, kv_heads, head_dim, block_size]
    k_scales: torch.Tensor    # fp32 [num_blocks, kv_heads]
    v_scales: torch.Tensor    # fp32 [num_blocks, kv_heads]

    @classmethod
    def empty(cls, num_blocks: int, kv_heads: int, head_dim: int, block_size: int = 64, device="cuda"):
        codes = lambda *shape: torch.zeros(num_blocks, kv_heads, *shape, dtype=torch.int8, device=device)
        scales = lambda: torch.zeros(num_blocks, kv_heads, dtype=torch.float32, device=device)
        return cls(codes(block_size, head_dim), codes(head_dim, block_size), scales(), scales())

    def _sizes(self):
        k, v, ks, vs = self
        nb, h, bs, d = k.shape
        if (v.shape != (nb, h, d, bs) or ks.shape != (nb, h) or vs.shape != (nb, h) or k.dtype != torch.int8
                or v.dtype != torch.int8 or ks.dtype != torch.float32 or vs.dtype != torch.float32
                or not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous())):
            raise ValueError("cache tensors must be contiguous: int8 k [blocks, heads, block_size, dim] and v "
                             "[blocks, heads, dim, block_size], fp32 scales [blocks, heads]")
        for t, name in zip(self, ("cache.k", "cache.v", "cache.k_scales", "cache.v_scales")):
            _on_gpu(t, name)
        return nb, h, d, bs


def _heads3(t, rows, heads, dim, name):
    """Row stride of a [rows, heads, dim] tensor whose heads follow each other."""
    if t.shape != (rows, heads, dim):
        raise ValueError(f"{name} must be {(rows, heads, dim)}, got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != dim):
        raise ValueError(f"{name}: the heads of a row must follow each other")
    _on_gpu(t, name)
    return s0 if rows > 1 else heads * dim


def _ragged(offsets, starts, block_table, name):
    batch = starts.numel()
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, width]")
    return (_vector(offsets, batch + 1, torch.int32, "offsets"), _vector(starts, batch, torch.int32, name), batch,
            _vector(block_table, block_table.numel(), torch.int32, "block_table"), block_table.shape[1])


def kv_cache_write_int8(cache: KVCacheInt8, K, V, offsets, starts, block_table):
    """kv_cache_write_int8 (include/ptq.h): quantize K, V [rows, kv_heads, head_dim] into the cache, rows
    offsets[b] .. offsets[b + 1] at positions starts[b], ... of sequence b."""
    nb, h, d, bs = cache._sizes()
    rows = K.shape[0]
    ldk, ldv = _heads3(K, rows, h, d, "K"), _heads3(V, rows, h, d, "V")
    if V.dtype != K.dtype:
        raise TypeError("K and V must have one dtype")
    _check(_lib.kv_cache_write_int8(_ptr(cache.k), _ptr(cache.v), _ptr(cache.k_scales), _ptr(cache.v_scales), nb, h, d,
                                    bs, _ptr(K), ldk, _ptr(V), ldv, _dtype_code(K), rows,
                                    *_ragged(offsets, starts, block_table, "starts"), _stream()))


def kv_cache_read_int8(cache: KVCacheInt8, offsets, starts, block_table, rows: int, out_dtype=torch.bfloat16, K=None,
                       V=None):
    """kv_cache_read_int8 (include/ptq.h): (K, V) [rows, kv_heads, head_dim] of the same ragged rows."""
    nb, h, d, bs = cache._sizes()
    if K is None:
        K = torch.empty(rows, h, d, dtype=out_dtype, device=cache.k.device)
    if V is None:
        V = torch.empty(rows, h, d, dtype=K.dtype, device=cache.k.device)
    ldk, ldv = _heads3(K, rows, h, d, "K"), _heads3(V, rows, h, d, "V")
    if V.dtype != K.dtype:
        raise TypeError("K and V must have one dtype")
    _check(_lib.kv_cache_read_int8(_ptr(cache.k), _ptr(cache.v), _ptr(cache.k_scales), _ptr(cache.v_scales), nb, h, d,
                                   bs, _ptr(K), ldk, _ptr(V), ldv, _dtype_code(K), rows,
                                   *_ragged(offsets, starts, block_table, "starts"), _stream()))
    return K, V


def attention_int8_cache_workspace_bytes(rows: int, batch: int, heads: int, kv_heads: int, head_dim: int,
                                         block_size: int, table_width: int) -> int:
    return int(_lib.attention_int8_cache_workspace_bytes(rows, batch, heads, kv_heads, head_dim, block_size,
                                                         table_width))


def attention_int8_cache(Q, cache: KVCacheInt8, offsets, seq_lens, block_table, scale=None, causal=True, window=0,
                         O=None, lse=None, return_lse=False, workspace=None):
    """attention_int8_cache (include/ptq.h): attention of Q [rows, heads, head_dim] over the cache; seq_lens counts
    each sequence's keys, the call's own tokens included. Returns O, or (O, lse) with return_lse or a given lse."""
    nb, h, d, bs = cache._sizes()
    rows, heads = Q.shape[0], Q.shape[1]
    if scale is None:
        scale = d ** -0.5
    if O is None:
        O = torch.empty(rows, heads, d, dtype=Q.dtype, device=Q.device)
    if lse is None and return_lse:
        lse = torch.empty(rows, heads, dtype=torch.float32, device=Q.device)
    ldq, ldo = _heads3(Q, rows, heads, d, "Q"), _heads3(O, rows, heads, d, "O")
    if O.dtype != Q.dtype:
        raise TypeError("O must have Q's dtype")
    off, lens, batch, table, width = _ragged(offsets, seq_lens, block_table, "seq_lens")
    ws, wsb = _scratch(attention_int8_cache_workspace_bytes(rows, batch, heads, h, d, bs, width), Q.device, workspace)
    _check(_lib.attention_int8_cache(_ptr(Q), ldq, _ptr(O), ldo, _vector(lse, rows * heads, torch.float32, "lse"),
                                     _dtype_code(Q), rows, heads, off, lens, batch, table, width, _ptr(cache.k),
                                     _ptr(cache.v), _ptr(cache.k_scales), _ptr(cache.v_scales), nb, h, d, bs,
                                     float(scale), int(bool(causal)), window, _ptr(ws), wsb, _stream()))
    return O if lse is None else (O, lse)


# ------------------------------------------------------------- test hook ---

def _test_gemm_f32(A, B, C, M, N, K, layout_a, layout_b, alpha=1.0, beta_one=0, tri=0, upper_only=0):
    """ptq_test_gemm_f32 (include/ptq_testing.h): the fp32 MFMA GEMM alone."""
    _check(_lib.ptq_test_gemm_f32(M, N, K, _ptr(A), A.stride(0), layout_a, _ptr(B), B.stride(0), layout_b, _ptr(C),
                                  C.stride(0), float(alpha), int(beta_one), int(tri), int(upper_only), _stream()))
    return C


def _test_gemm_f32_pair(p0, p1):
    """ptq_test_gemm_f32_pair (include/ptq_testing.h): two products in one launch, the first with B stored
    [N][K], the second with B row-major [K][N]. Each pi is a dict with A, B, C, M, N, K and optionally alpha,
    beta_one, tri, upper_only."""
    def args(p):
        return (p["M"], p["N"], p["K"], _ptr(p["A"]), p["A"].stride(0), _ptr(p["B"]), p["B"].stride(0), _ptr(p["C"]),
                p["C"].stride(0), float(p.get("alpha", 1.0)), int(p.get("beta_one", 0)), int(p.get("tri", 0)),
                int(p.get("upper_only", 0)))
    _check(_lib.ptq_test_gemm_f32_pair(*args(p0), *args(p1), _stream()))


def _test_gemm_f32_split3(A, B, C, M, N, K, layout_a, layout_b, alpha=1.0, beta_one=0, tri=0, upper_only=0):
    """ptq_test_gemm_f32_split3 (include/ptq_testing.h): the same product on the bf16 MFMA from split operands."""
    ws, wsb = _workspace(int(_lib.ptq_test_gemm_f32_split3_workspace_bytes(M, N, K)), C.device, None)
    _check(_lib.ptq_test_gemm_f32_split3(M, N, K, _ptr(A), A.stride(0), layout_a, _ptr(B), B.stride(0), layout_b,
                                         _ptr(C), C.stride(0), float(alpha), int(beta_one), int(tri),
                                         int(upper_only), _ptr(ws), wsb, _stream()))
    return C


def _test_matmul_int8_plan(rows, out, n):
    """ptq_test_matmul_int8_plan (include/ptq_testing.h): (shape, nsplit) that matmul_int8 chooses."""
    shape, nsplit = ctypes.c_int(), ctypes.c_int()
    _check(_lib.ptq_test_matmul_int8_plan(rows, out, n, ctypes.byref(shape), ctypes.byref(nsplit)))
    return shape.value, nsplit.value


def _test_matmul_int8(shape, nsplit, A, a_scales, codes, scales, bias=None, out_dtype=torch.bfloat16, Y=None):
    """ptq_test_matmul_int8 (include/ptq_testing.h): matmul_int8 by the kernel that shape and nsplit name."""
    rows, n = A.shape
    out = codes.shape[0]
    Y, ldy = _product_output(Y, rows, out, out_dtype, A.device)
    ws, wsb = _workspace(int(_lib.ptq_test_matmul_int8_workspace_bytes(shape, nsplit, rows, out, n)), A.device, None)
    _check(_lib.ptq_test_matmul_int8(shape, nsplit, _ptr(A), _codes(A, "A"),
                                     _vector(a_scales, rows, torch.float32, "a_scales"), rows, _ptr(codes),
                                     _codes(codes, "codes"), _vector(scales, out, torch.float32, "scales"), out, n,
                                     _vector(bias, out, torch.float32, "bias"), _dtype_code(Y), _ptr(Y), ldy, _ptr(ws),
                                     wsb, _stream()))
    return Y


def _test_attention_int8_plan(rows, batch, heads, kv_heads, head_dim, block_size, table_width, window=0):
    """ptq_test_attention_int8_plan (include/ptq_testing.h): (tiles, waves, nsplit) that attention_int8_cache chooses."""
    plan = [ctypes.c_int() for _ in range(3)]
    _check(_lib.ptq_test_attention_int8_plan(rows, batch, heads, kv_heads, head_dim, block_size, table_width, window,
                                             *map(ctypes.byref, plan)))
    return tuple(x.value for x in plan)


def _test_attention_int8_cache(tiles, waves, nsplit, Q, cache, offsets, seq_lens, block_table, scale=None, causal=True,
                               window=0):
    """ptq_test_attention_int8_cache (include/ptq_testing.h): (O, lse) by the kernel that the first three name."""
    nb, h, d, bs = cache._sizes()
    rows, heads = Q.shape[0], Q.shape[1]
    O = torch.empty(rows, heads, d, dtype=Q.dtype, device=Q.device)
    lse = torch.empty(rows, heads, dtype=torch.float32, device=Q.device)
    off, lens, batch, table, width = _ragged(offsets, seq_lens, block_table, "seq_lens")
    ws, wsb = _workspace(int(_lib.ptq_test_attention_int8_workspace_bytes(nsplit, rows, heads, d)), Q.device, None)
    _check(_lib.ptq_test_attention_int8_cache(int(tiles), waves, nsplit, _ptr(Q), _heads3(Q, rows, heads, d, "Q"),
                                              _ptr(O), heads * d, _ptr(lse), _dtype_code(Q), rows, heads, off, lens,
                                              batch, table, width, _ptr(cache.k), _ptr(cache.v), _ptr(cache.k_scales),
                                              _ptr(cache.v_scales), nb, h, d, bs, float(scale or d ** -0.5),
                                              int(bool(causal)), window, _ptr(ws), wsb, _stream()))
    return O, lse
