"""GPU: rotary_apply from some columns of a projection's rows into others of the same rows, before them and behind them."""
import pytest
import torch

from gpu_util import announce
from test_gpu_14_kv_cache_int8 import _ints, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,x,y", [(5, 0, 3), (5, 3, 0), (5, 2, 5), (1, 0, 3), (400, 4, 1), (3, 5, 2)])
def test_other_columns_of_the_same_rows(gpu, rows, x, y, dtype):
    from post_int4_weight_amd import api
    announce(f"rotary of heads {x} .. {x + 3} into {y} .. {y + 3} of {rows} rows {dtype}")
    rotary = api.Rotary.make(48, device=gpu)
    wide, pos = _rows(rows, 8, 64, dtype, gpu, rows), _ints(range(7, rows + 7), gpu)
    want = wide.clone()
    want[:, y:y + 3] = api.rotary_apply(wide[:, x:x + 3].contiguous(), rotary, pos)
    api.rotary_apply(wide[:, x:x + 3], rotary, pos, Y=wide[:, y:y + 3])
    torch.cuda.synchronize()
    assert torch.equal(wide, want)
