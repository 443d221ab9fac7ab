"""GPU: int8 linear operators at sizes past what one launch takes (2^32 threads). The inputs repeat, so that the outputs of
the whole are those of a part."""
import pytest
import torch

from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_quantize_tokens_many_rows(gpu):
    from post_int4_weight_amd import api
    rows, n, part = (1 << 24) + 40, 8, 1 << 20
    announce(f"quantize_tokens_int8 rows={rows} in={n}")
    X = torch.randn(part, n, generator=torch.Generator().manual_seed(1)).bfloat16().to(gpu)
    codes, scales = api.quantize_tokens_int8(X)
    big = X.repeat(rows // part + 1, 1)[:rows]
    got, s = api.quantize_tokens_int8(big)
    torch.cuda.synchronize()
    for r in range(0, rows, part):
        m = min(part, rows - r)
        assert torch.equal(got[r:r + m], codes[:m]) and torch.equal(s[r:r + m], scales[:m]), r


@pytest.mark.parametrize("rows,out,n", [(65536 + 24, 16384 + 40, 8), (3, (1 << 26) + 72, 8), (20, (1 << 26) + 72, 8)])
def test_products_of_many_outputs(gpu, rows, out, n):
    """Depths below one stage go through workgroups of 16 x 16 outputs and 1024 threads, however many outputs there are."""
    from post_int4_weight_amd import api
    announce(f"linear_int8 and matmul_int8 rows={rows} out={out} in={n}")
    gen = torch.Generator().manual_seed(2)
    some, few = min(rows, 40), min(out, 4096)
    X = torch.randn(some, n, generator=gen).bfloat16().to(gpu)
    W = torch.randint(-128, 128, (few, n), generator=gen, dtype=torch.int8).to(gpu)
    sw, bias = (torch.rand(few, generator=gen) + 0.5).to(gpu), torch.randn(few, generator=gen).to(gpu)
    want = api.linear_int8(X, W, sw, bias)
    over = lambda t, m: t.repeat(m // t.shape[0] + 1, *[1] * (t.dim() - 1))[:m].contiguous()
    big_W, big_sw, big_bias = over(W, out), over(sw, out), over(bias, out)
    big_X = over(X, rows)
    A, sa = api.quantize_tokens_int8(big_X)
    for Y in (api.linear_int8(big_X, big_W, big_sw, big_bias), api.matmul_int8(A, sa, big_W, big_sw, big_bias)):
        torch.cuda.synchronize()
        for r in range(0, rows, some):
            m = min(some, rows - r)
            if rows > 100 and r % 4000 and r + 8 * some < rows:
                continue                         # every hundredth stretch, and the last ones
            for o in range(0, out, few):
                k = min(few, out - o)
                assert torch.equal(Y[r:r + m, o:o + k], want[:m, :k]), (r, o)
        del Y
