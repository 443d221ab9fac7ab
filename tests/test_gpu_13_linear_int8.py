"""GPU: the int8 linear layer (quantize_tokens_int8, matmul_int8, linear_int8)
against the fp64 oracle (oracle/int8.py).

Bounds. Scales: one correctly rounded fp32 division, so equal. Codes: equal to
rint(x / S) except within oracle.int8.code_slack of a tie (roundings of S,
1 / S, the product; one more for x / s). Products: the int32 sums are exact, so
from the same codes Y differs from fp64 by the roundings of (float)sum, sx sw
and their product (3 u |y - bias|), of the bias sum (u |y|) and of the output
(half a step of 8 significant bits: 2^-8 |y| for bf16).
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import int8 as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _x(rows, n, dtype, gpu, seed):
    gen = torch.Generator().manual_seed(seed)
    sigma = torch.exp(torch.randn(n, generator=gen))
    return (torch.randn(rows, n, generator=gen) * sigma).to(DTYPES[dtype]).to(gpu), sigma.sqrt().to(gpu)


def _w(out, n, gpu, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randint(-128, 128, (out, n), generator=gen, dtype=torch.int8).to(gpu),
            (torch.rand(out, 1, generator=gen) + 0.5).to(gpu) / 1000)


def _check_product(Y, A, sa, W, sw, bias, name):
    b = None if bias is None else bias.cpu().double().numpy()
    want = ref.matmul(A.cpu().numpy(), sa.cpu().double().numpy(), W.cpu().numpy(), sw.cpu().double().numpy(), b)
    raw = want if b is None else want - b
    tol = 3 * ref.U * np.abs(raw) + ref.U * np.abs(want) + 1e-37
    if Y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8)
    err = np.abs(to64(Y) - want)
    assert np.all(err <= tol * 1.01), (name, float((err / tol).max()))


@pytest.mark.parametrize("rows,n,dtype,smooth", [(1, 8, "bf16", False), (3, 64, "f32", True), (5, 1000, "bf16", True),
                                                 (2, 4096, "bf16", False), (4, 8200, "f32", False),
                                                 (2, 16392, "bf16", True), (3, 40008, "bf16", False)])
def test_quantize_tokens(gpu, rows, n, dtype, smooth):
    from post_int4_weight_amd import api
    announce(f"quantize_tokens_int8 rows={rows} in={n} {dtype} smooth={smooth}")
    X, s = _x(rows, n, dtype, gpu, n)
    codes, scales = api.quantize_tokens_int8(X, s if smooth else None)
    torch.cuda.synchronize()
    x = to64(X)
    if smooth:   # x / s is an fp32 number by definition
        x = (x.astype(np.float32) / s.cpu().numpy()).astype(np.float64)
    quot, S = ref.quantize_tokens(x)
    assert np.array_equal(to64(scales), S)
    assert ref.codes_agree(codes.cpu().numpy(), quot, ref.code_slack())


def test_quantize_tokens_zero_tiny_and_non_finite_rows(gpu):
    from post_int4_weight_amd import api
    announce("quantize_tokens_int8: zero, tiny, NaN and infinite rows")
    X = torch.randn(6, 72, generator=torch.Generator().manual_seed(1)).to(gpu)
    X[0] = 0
    X[1] *= 1e-38 / X[1].abs().max()     # scale below FLT_MIN: stored as 0
    X[2, 70] = float("nan")
    X[3, 0] = float("inf")
    X[4] *= 3e38 / X[4].abs().max()
    codes, scales = api.quantize_tokens_int8(X)
    Y = api.matmul_int8(codes, scales, torch.ones(5, 72, dtype=torch.int8, device=gpu), torch.ones(5, device=gpu))
    torch.cuda.synchronize()
    S = to64(scales)
    assert S[0] == 0 and S[1] == 0 and np.isnan(S[2]) and np.isnan(S[3]) and np.isfinite(S[4:]).all()
    assert not codes[:2].any() and int(codes[4].abs().max()) == 127
    y = to64(Y)
    assert (y[:2] == 0).all() and np.isnan(y[2:4]).all() and np.isfinite(y[4:]).all()


SIZES = [(1, 1, 8), (1, 4096, 4096), (1, 1000, 136), (2, 17, 1000), (5, 130, 72), (16, 256, 2056), (17, 512, 1024),
         (33, 100, 14336), (48, 1024, 512), (64, 320, 4104), (65, 64, 256), (129, 257, 640), (200, 1000, 1032),
         (256, 256, 128), (300, 512, 384), (513, 129, 4096), (1000, 2048, 256)]


@pytest.mark.parametrize("rows,out,n", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matmul(gpu, rows, out, n, dtype):
    from post_int4_weight_amd import api
    announce(f"matmul_int8 rows={rows} out={out} in={n} {dtype}")
    gen = torch.Generator().manual_seed(rows)
    A = torch.randint(-128, 128, (rows, n), generator=gen, dtype=torch.int8).to(gpu)
    sa = (torch.rand(rows, generator=gen) + 0.1).to(gpu)
    W, sw = _w(out, n, gpu, out)
    bias = torch.randn(out, generator=gen).to(gpu) if rows % 2 else None
    Y = api.matmul_int8(A, sa, W, sw, bias=bias, out_dtype=DTYPES[dtype])
    again = api.matmul_int8(A, sa, W, sw, bias=bias, out_dtype=DTYPES[dtype])
    torch.cuda.synchronize()
    _check_product(Y, A, sa, W, sw, bias, (rows, out, n))
    assert torch.equal(Y, again)


@pytest.mark.parametrize("rows,out,n,pad", [(3, 40, 1000, 8), (40, 200, 264, 24), (300, 300, 520, 40),
                                            (300, 512, 512, 16)])
def test_matmul_row_strides(gpu, rows, out, n, pad):
    """Operands and output are column ranges of wider tensors; what is around the output stays."""
    from post_int4_weight_amd import api
    announce(f"matmul_int8 strided rows={rows} out={out} in={n} pad={pad}")
    gen = torch.Generator().manual_seed(7)
    wide = lambda r: torch.randint(-128, 128, (r, n + pad), generator=gen, dtype=torch.int8).to(gpu)
    A, W = wide(rows)[:, :n], wide(out)[:, :n]
    sa, sw = torch.rand(rows, generator=gen).to(gpu), torch.rand(out, generator=gen).to(gpu)
    big = torch.full((rows + 6, out + 5), 7.0, device=gpu)
    Y = big[4:4 + rows, :out]
    api.matmul_int8(A, sa, W, sw, Y=Y)
    torch.cuda.synchronize()
    _check_product(Y, A, sa, W, sw, None, (rows, out, n))
    Y.fill_(7.0)
    assert torch.all(big == 7.0)


@pytest.mark.parametrize("rows,out,n,dtype,smooth", [(1, 512, 1024, "bf16", False), (1, 33, 4104, "f32", True),
                                                     (7, 257, 1000, "f32", True), (37, 128, 28672, "bf16", False),
                                                     (130, 300, 264, "bf16", True), (515, 1024, 2048, "bf16", True)])
def test_linear(gpu, rows, out, n, dtype, smooth):
    """linear_int8 is its two halves, bit for bit, and near the fp64 product of the unquantized activations."""
    from post_int4_weight_amd import api
    announce(f"linear_int8 rows={rows} out={out} in={n} {dtype} smooth={smooth}")
    X, s = _x(rows, n, dtype, gpu, rows + n)
    s = s if smooth else None
    W, sw = _w(out, n, gpu, n)
    bias = torch.randn(out, generator=torch.Generator().manual_seed(3)).to(gpu)
    Y = api.linear_int8(X, W, sw, bias=bias, s=s)
    codes, scales = api.quantize_tokens_int8(X, s)
    halves = api.matmul_int8(codes, scales, W, sw, bias=bias, out_dtype=X.dtype)
    torch.cuda.synchronize()
    assert Y.dtype == X.dtype and torch.equal(Y, halves)
    _check_product(Y, codes, scales, W, sw, bias, (rows, out, n))
    # against unquantized activations: half a step of every code at most
    x = to64(X) / (1.0 if s is None else to64(s))
    w = W.cpu().double().numpy() * to64(sw)
    exact = x @ w.T + to64(bias)
    step = 0.5 * (1 + 1e-4) * to64(scales)[:, None] * np.abs(w).sum(1)[None, :]
    assert np.all(np.abs(to64(Y) - exact) <= step + 2.0 ** -8 * np.abs(exact) + 1e-5)


def test_linear_of_a_gptq_layer(gpu):
    """Per-channel 8-bit codes from the quantizer go in as they are; the error is quantization error."""
    import inputs
    from gpu_util import zeros_h
    from post_int4_weight_amd import api
    announce("linear_int8 on gptq_quantize_layer's codes (8 bits, one group, act-order)")
    W, X = inputs.custom(384, 512, 4096, 5, "bf16", gpu)
    H, d = zeros_h(512, gpu)
    api.hessian_accumulate(H, d, X)
    res = api.gptq_quantize_layer(W, H, d, bits=8, group_size=512, act_order=True)
    Y = api.linear_int8(X[:257], res["codes"], res["scales"])
    torch.cuda.synchronize()
    want = to64(X[:257]) @ to64(W).T
    # 8-bit codes on both sides: steps of 2 amax / 254, amax about 4 rms: 0.9% of rms each, uniform error / sqrt(3);
    # outlier channels make rows' amax up to about ten times that
    assert np.linalg.norm(to64(Y) - want) / np.linalg.norm(want) < 0.05


def test_empty_and_other_stream(gpu):
    from post_int4_weight_amd import api
    announce("linear_int8: no rows, no outputs; work on another stream")
    W, sw = _w(24, 64, gpu, 1)
    assert api.linear_int8(torch.empty(0, 64, device=gpu), W, sw).shape == (0, 24)
    assert api.linear_int8(torch.ones(3, 64, device=gpu), W[:0], sw[:0]).shape == (3, 0)
    X, _ = _x(70, 64, "f32", gpu, 2)
    want = api.linear_int8(X, W, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = api.linear_int8(X * 1.0, W, sw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_graph_replay(gpu):
    """Captured once, replayed on new inputs with eager work between the replays."""
    from post_int4_weight_amd import api
    announce("linear_int8 in a captured graph")
    for rows in (1, 40, 300):
        W, sw = _w(512, 2048, gpu, 4)
        X = torch.zeros(rows, 2048, dtype=torch.bfloat16, device=gpu)
        Y = torch.empty(rows, 512, dtype=torch.bfloat16, device=gpu)
        ws = torch.empty(max(1, api.linear_int8_workspace_bytes(rows, 512, 2048)), dtype=torch.uint8, device=gpu)
        api.linear_int8(X, W, sw, Y=Y, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.linear_int8(X, W, sw, Y=Y, workspace=ws)
        for k in range(4):
            X.copy_(_x(rows, 2048, "bf16", gpu, k)[0])
            graph.replay()
            got = Y.clone()
            want = api.linear_int8(X, W, sw)
            torch.cuda.synchronize()
            assert torch.equal(got, want), (rows, k)


def test_refusals(gpu):
    from post_int4_weight_amd import api
    X, W, sw = torch.ones(4, 64, device=gpu), torch.ones(8, 64, dtype=torch.int8, device=gpu), torch.ones(8, device=gpu)
    with pytest.raises(ValueError):
        api.linear_int8(X[:, :56], W, sw)                        # widths differ
    with pytest.raises(ValueError):
        api.linear_int8(X, W, sw[:5])                            # scales per output channel
    with pytest.raises(TypeError):
        api.linear_int8(X, W.float(), sw)
    with pytest.raises(TypeError):
        api.linear_int8(X.double(), W, sw)
    with pytest.raises(ValueError):
        api.linear_int8(X.t(), W[:, :4], sw)                     # not row-major
    with pytest.raises(api.PTQError) as e:
        api.linear_int8(X[:, :60], W[:, :60], sw)                # in % 8
    assert e.value.name == "PTQ_EINVAL" and "multiple of 8" in str(e.value)
    with pytest.raises(api.PTQError) as e:
        api.linear_int8(X, W, sw, workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
    assert e.value.name == "PTQ_EWORKSPACE"
