"""fp64 oracle of the int8 serving operators: activations quantized per token,
the int8 linear product, the int8 block cache and attention over it.

Written from the definitions, sequence by sequence and block by block. Scales
are fp32 numbers by definition (S = a / 127 rounded to fp32); everything else
is fp64. A code is rint(x / S): ``code_slack`` says how near a tie the fp32
evaluation x * (1 / S) may decide otherwise.
"""
from __future__ import annotations

import numpy as np

FLT_MIN = float(np.finfo(np.float32).tiny)
U = 2.0 ** -24          # unit roundoff of fp32


def scale_of(a) -> np.ndarray:
    """fp32 scale (as float64) of sets with largest magnitude a."""
    a = np.asarray(a, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        s = (a.astype(np.float32) / np.float32(127)).astype(np.float64)
    s = np.where(s < FLT_MIN, 0.0, s)
    return np.where(np.isfinite(a), s, np.nan)


def quotient(x, s):
    """x / s with 0 where the scale is 0."""
    return np.divide(x, s, out=np.zeros(np.broadcast(x, s).shape), where=np.asarray(s) > 0)


def code_slack(extra: int = 0) -> float:
    """|x (1/S) - x/S| in code steps: roundings of S, 1/S and the product (and `extra` more) at 127 steps."""
    return (3 + extra) * U * 127 * 1.01


def codes_agree(codes, quot, slack) -> bool:
    """codes == rint(quot), or quot within slack of the half between the two."""
    codes = np.asarray(codes, dtype=np.float64)
    return bool(np.all(np.abs(codes - quot) <= 0.5 + slack)) and bool(np.all(np.abs(codes) <= 127))


def quantize_tokens(x, s=None):
    """(x / s) / S per row [rows, in] (unrounded codes), S [rows]."""
    x = np.asarray(x, dtype=np.float64)
    if s is not None:
        x = x / np.asarray(s, dtype=np.float64)
    S = scale_of(np.abs(x).max(axis=1))
    return quotient(x, S[:, None]), S


def matmul(a, sa, w, sw, bias=None):
    y = (np.asarray(a, np.float64) @ np.asarray(w, np.float64).T) * np.asarray(sa, np.float64)[:, None]
    y = y * np.asarray(sw, np.float64).reshape(1, -1)
    return y if bias is None else y + np.asarray(bias, np.float64)


class Cache:
    """Codes [num_blocks, heads, bs, dim] and scales of both halves, filled by the calls of write(). near marks the
    codes whose unrounded value was within code_slack of a tie, now or before a recoding: fp32 may decide it the other
    way (bf16 values make exact ties common, as of c 3/4 when a scale grows by 4/3)."""

    def __init__(self, num_blocks, heads, dim, bs):
        self.bs = bs
        self.codes = {h: np.zeros((num_blocks, heads, bs, dim)) for h in "kv"}
        self.scales = {h: np.zeros((num_blocks, heads)) for h in "kv"}
        self.near = {h: np.zeros((num_blocks, heads, bs, dim), dtype=bool) for h in "kv"}

    def write(self, half, x, offsets, starts, table):
        """x [rows, heads, dim] of the ragged rows (offsets, starts, table: lists)."""
        bs, codes, scales, near = self.bs, self.codes[half], self.scales[half], self.near[half]
        tie = lambda q: np.abs(np.abs(q - np.rint(q)) - 0.5) <= code_slack()
        for b, start in enumerate(starts):
            n = offsets[b + 1] - offsets[b]
            at = start
            while at < start + n:
                block, end = table[b][at // bs], min((at // bs + 1) * bs, start + n)
                rows = np.asarray(x[offsets[b] + at - start:offsets[b] + end - start], np.float64)
                for h in range(codes.shape[1]):
                    S = float(scale_of(np.abs(rows[:, h]).max()))
                    held = at % bs
                    if held:
                        old = scales[block, h]
                        if S > old:
                            q = codes[block, h, :held] * (old / S)
                            codes[block, h, :held] = np.rint(q)
                            near[block, h, :held] |= tie(q)
                        S = max(S, old)
                    scales[block, h] = S
                    q = quotient(rows[:, h], S)
                    codes[block, h, held:held + end - at] = np.rint(q)
                    near[block, h, held:held + end - at] = tie(q)
                at = end


def attention(q, k, v, scale, pos0, causal=True, window=0):
    """One sequence and head: q [n, d], k and v [len, d] in fp64, query i at position pos0 + i. Returns o, lse and
    what error bounds need: A = sum w|v| / sum w, B = the largest sum_d |q k| scale and C = the largest |logit| of the
    row's keys, N = its number of keys."""
    n, length = q.shape[0], k.shape[0]
    o, lse = np.zeros((n, q.shape[1])), np.full(n, -np.inf)
    A, B, C, N = np.zeros_like(o), np.zeros(n), np.zeros(n), np.zeros(n, dtype=np.int64)
    for i in range(n):
        p = pos0 + i
        lo = max(0, p - window + 1) if window else 0
        hi = min(p + 1, length) if causal else length
        if hi <= lo:
            continue
        t = scale * (k[lo:hi] @ q[i])
        w = np.exp(t - t.max())
        o[i], lse[i] = w @ v[lo:hi] / w.sum(), t.max() + np.log(w.sum())
        A[i], N[i] = w @ np.abs(v[lo:hi]) / w.sum(), hi - lo
        B[i], C[i] = abs(scale) * (np.abs(k[lo:hi]) @ np.abs(q[i])).max(), np.abs(t).max()
    return o, lse, A, B, C, N
