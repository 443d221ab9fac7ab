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
