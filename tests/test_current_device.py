"""A launch goes to the current device: operands on another one are refused by the int8 serving operators and those of drafted
tokens. Needs no GPU: the devices are made up."""
import inspect
import re

import pytest
import torch

from post_int4_weight_amd import api

OPERATORS = [api.quantize_tokens_int8, api.matmul_int8, api.linear_int8, api.kv_cache_write_int8, api.kv_cache_read_int8,
             api.attention_int8_cache, api.rotary_apply, api.kv_cache_append_int8, api.attention_int8_tree, api._verify]


class On:
    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


def test_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    assert api._stream() == 101 and api._stream(On(1)) == 101
    for other in (0, 2):
        with pytest.raises(ValueError, match=f"tensors on cuda:{other}, but the current device is cuda:1"):
            api._stream(On(other))


@pytest.mark.parametrize("operator", OPERATORS, ids=lambda f: f.__name__)
def test_operators_name_an_operand(operator):
    """The stream that an operator takes is asked for with one of its operands."""
    asked = re.findall(r"_stream\(([\w.]*)\)", inspect.getsource(operator))
    known = set(inspect.signature(operator).parameters)
    assert asked and all(name.split(".")[0] in known for name in asked), asked
