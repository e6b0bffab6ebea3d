"""Tensors on another device than the current one are refused: the C library launches on the current
device (the header's convention for every pointer), whose kernels cannot reach them."""
import types

import pytest
import torch

import ternary_weight_linear_amd as tw


def on(index):
    return types.SimpleNamespace(device=torch.device("cuda", index))


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(tw, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match=r"cuda:1, but the current device is cuda:0.*torch.cuda.device\(1\)"):
        tw._dev(on(1), on(1))
    with pytest.raises(ValueError, match="one device"):
        tw._dev(on(0), on(1))
    assert tw._dev(on(0), None, on(0)) == torch.device("cuda", 0)
    monkeypatch.setattr(tw, "_current_device", lambda: 1)
    assert tw._dev(on(1)) == torch.device("cuda", 1)


@pytest.mark.parametrize("call", [n for n in sorted(tw.__all__) if isinstance(getattr(tw, n), types.FunctionType)])
def test_every_entry_point_with_tensors_checks_their_device(call):
    code = getattr(tw, call).__code__
    if "_stream" in code.co_names:
        assert "_dev" in code.co_names
