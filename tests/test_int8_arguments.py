"""Arguments that the Python entry points of the int8 serving operators refuse before anything reaches the GPU."""
import pytest
import torch

from post_int4_weight_amd import api


def _codes(*shape):
    return torch.zeros(*shape, dtype=torch.int8)


@pytest.mark.parametrize("rows", [1, 3])
def test_output_columns_follow_each_other(rows):
    """Y of one row, too: its columns are written one after another, whatever its strides say."""
    A, sa, W, sw = _codes(rows, 64), torch.ones(rows), _codes(8, 64), torch.ones(8)
    for Y in (torch.empty(8, 2 * rows)[:, :rows].t(), torch.empty(rows, 1).expand(rows, 8),
              torch.empty(rows, 16)[:, ::2]):
        with pytest.raises(ValueError, match="Y must be a 2-D row-major"):
            api.matmul_int8(A, sa, W, sw, Y=Y)
        with pytest.raises(ValueError, match="Y must be a 2-D row-major"):
            api.linear_int8(torch.zeros(rows, 64), W, sw, Y=Y)


def test_tensors_on_the_host_are_refused():
    """The GPU would fault on a host address: whichever argument it is, the call says so first."""
    rows, n, out, heads, dim, bs = 3, 64, 8, 2, 64, 16
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    X, A, W = torch.zeros(rows, n), _codes(rows, n), _codes(out, n)
    refused = lambda name: pytest.raises(ValueError, match=f"{name} must be on the GPU, not on cpu")
    with refused("X"):
        api.quantize_tokens_int8(X)
    with refused("A"):
        api.matmul_int8(A, torch.ones(rows), W, torch.ones(out))
    with refused("X"):
        api.linear_int8(X, W, torch.ones(out))
    cache = api.KVCacheInt8.empty(4, heads, dim, bs, device="cpu")
    K = torch.zeros(rows, heads, dim)
    with refused("cache.k"):
        api.kv_cache_write_int8(cache, K, K, ints(2), ints(1), ints(1, 1))
    with refused("cache.k"):
        api.kv_cache_read_int8(cache, ints(2), ints(1), ints(1, 1), rows)
    with refused("cache.k"):
        api.attention_int8_cache(K, cache, ints(2), ints(1), ints(1, 1))
    # each helper that an argument goes through
    for call in (lambda: api._vector(ints(2), 2, torch.int32, "offsets"), lambda: api._codes(A, "A"),
                 lambda: api._heads3(K, rows, heads, dim, "Q"), lambda: api._ragged(ints(2), ints(1), ints(1, 1), "starts"),
                 lambda: api._scratch(16, "cpu", torch.zeros(16, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="must be on the GPU, not on cpu"):
            call()
