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
