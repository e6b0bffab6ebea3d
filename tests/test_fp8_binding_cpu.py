"""Refusals of the binding's 8-bit floating point calls that are seen before any device is used."""
import pytest
import torch

import ternary_weight_linear_amd as tw

x = torch.zeros(4, 256, dtype=torch.float16)
w, s = torch.zeros(100, 256, dtype=torch.float8_e4m3fn), torch.zeros(1, 2)
q, sx = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(2, 4)
index, weight = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
wgu, sgu = torch.zeros(8, 2, 128, 256, dtype=torch.float8_e4m3fn), torch.zeros(8, 2, 1, 2)
wd, sd = torch.zeros(8, 256, 128, dtype=torch.float8_e4m3fn), torch.zeros(8, 2, 1)
CALLS = {"linear": lambda **kw: tw.bl_fp8_linear(q, sx, w, s, **kw), "forward": lambda **kw: tw.bl_fp8_forward(x, w, s, **kw),
         "experts": lambda **kw: tw.bl_fp8_experts(x, index, weight, wgu, sgu, wd, sd, **kw)}


@pytest.mark.parametrize("name", list(CALLS))
def test_out_of_another_type_than_asked_for(name):
    out = torch.zeros(4, 256 if name == "experts" else 100, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="out must be torch.float32, got torch.bfloat16"):
        CALLS[name](out=out, out_dtype=torch.float32)
    for kw in (dict(out=out), dict(out=out, out_dtype=torch.bfloat16), dict(out_dtype=torch.float16), {}):
        with pytest.raises(ValueError, match="GPU"):   # the types agree: the next check is the device
            CALLS[name](**kw)


@pytest.mark.parametrize("name", list(CALLS))
def test_result_types_that_there_are_not(name):
    out = torch.zeros(4, 256 if name == "experts" else 100, dtype=torch.float64)
    for kw in (dict(out=out), dict(out_dtype=torch.float64), dict(out_dtype=torch.int32)):
        with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
            CALLS[name](**kw)
