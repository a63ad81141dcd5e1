"""The binding's checks of tensors on a machine without a GPU."""
import importlib.util
import os
import sys

import pytest
import torch

import routing_dispatch_expert_sigmoid_b200 as package
from routing_dispatch_expert_sigmoid_b200 import ops


@pytest.fixture
def ops_without_cuda(monkeypatch):
    """The binding as it is imported by a torch without a CUDA build."""
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    name = package.__name__ + ".ops_without_cuda"
    spec = importlib.util.spec_from_file_location(
        name, os.path.join(os.path.dirname(ops.__file__), "ops.py"))
    module = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, name, module)
    spec.loader.exec_module(module)
    return module


def test_host_tensors_are_refused_without_a_cuda_build(ops_without_cuda):
    o = ops_without_cuda
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(o.MoeError, match="x is on cpu"):
        o._arg("moe_norm", o._current(), "x", x, torch.bfloat16, 256)
    with pytest.raises(o.MoeError, match="x is on cpu"):
        o.moe_norm(o.norm_config(4, 64), x, h=torch.zeros_like(x))
    l, idx, w = torch.zeros(4, 64), torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4)
    with pytest.raises(o.MoeError, match="logits is on cpu"):
        o.moe_gate(o.gate_config(4, 64, 4), l, None, None, idx, w)
