"""The token operators' Python entry points: what they do around a call, without a GPU."""
import os
import re

import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "routed_expert_ffn_route_gb300")


@pytest.fixture(scope="module")
def native():
    moe.build()
    moe.lib()
    from routed_expert_ffn_route_gb300 import _tokens_native
    return _tokens_native


class Stream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device_index = handle, device


# -------------------------------------------------------------------- device and stream
@pytest.mark.parametrize("dev", [0, 1, 7])
def test_a_call_runs_with_its_operands_device_current(native, dev):
    """A default stream's handle is 0 on every device: the device has to be current."""
    assert native.trace(dev, None) == [f"current stream of {dev}", f"set {dev}", "call on 0",
                                       "restore"]
    assert native.trace(dev, Stream(0, dev)) == [f"set {dev}", "call on 0", "restore"]
    assert native.trace(dev, Stream(4096, dev)) == [f"set {dev}", "call on 4096", "restore"]


def test_a_stream_of_another_device_is_refused(native):
    for on, dev in [(0, 1), (1, 0)]:
        with pytest.raises(ValueError, match="device"):
            native.trace(dev, Stream(0, on))
    with pytest.raises(ValueError, match="CUDA device"):
        native.trace(-1, None)
    with pytest.raises(AttributeError):
        native.trace(0, object())


def test_every_entry_point_calls_through_the_device_guard():
    """Each C call of the extension module stands in the one function that sets the device."""
    with open(os.path.join(PKG, "csrc", "tokens_py.cpp")) as f:
        src = f.read()
    calls = re.findall(r"return (moe_\w+)\(", src)
    launched = re.findall(r"c\.launch\(a\[\d+\], \[&\]\(void \*st\) \{\s*return (moe_\w+)\(", src)
    assert sorted(calls) == sorted(launched) and len(calls) == 7
    assert "on_device<Cuda>" in src and "using Guard = c10::cuda::CUDAGuard;" in src


def test_a_torch_stream_says_its_device():
    """handle() reads these two attributes of torch.cuda.Stream."""
    assert hasattr(torch.cuda.Stream, "device_index") and hasattr(torch.cuda.Stream, "cuda_stream")
