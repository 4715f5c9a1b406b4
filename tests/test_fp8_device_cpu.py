"""FP8 calls on operands of a device that is not the current one: a launch goes
to the current device, so the binding makes the operands' device current for it
(the library's calls are replaced here, no GPU is needed)."""
import contextlib
import os
import re

import pytest
import torch

import microscaling_fp4_quantized_block_amd as mx
from microscaling_fp4_quantized_block_amd import fp8


class Devices:
    """A machine of several devices of which one is current; `seen` holds the current one at each library call."""

    def __init__(self, monkeypatch, current):
        self.current, self.seen = current, []
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(fp8, "_current_device", lambda: self.current, raising=False)
        monkeypatch.setattr(fp8, "_raw_stream", lambda index: 1000 + (index or 0))
        monkeypatch.setattr(torch.cuda, "device", self.made_current)
        monkeypatch.setattr(fp8, "lib", self)

    @contextlib.contextmanager
    def made_current(self, device):
        was, self.current = self.current, torch.device(device).index or 0
        yield
        self.current = was

    def mxfp4_fp8_dequantize(self, *args):
        self.seen.append((self.current, args[-1]))
        return 0


@pytest.mark.parametrize("current", [0, 1, 3])
def test_the_operands_device_is_current_for_the_launch(monkeypatch, current):
    q = mx.empty_fp8(4, 128, "cpu")
    q._device = torch.device("cuda", 0)   # (only its index is looked at)
    devices = Devices(monkeypatch, current)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))
    mx.mxfp4_fp8_dequantize(q)
    assert devices.seen == [(0, 1000)] and devices.current == current


def test_every_call_with_a_stream_goes_that_way():
    with open(os.path.join(os.path.dirname(mx.__file__), "fp8.py")) as f:
        text = f.read()
    assert len(re.findall(r"_raw_stream\(", text)) == 2   # (in _launch, for either case)
    for name in ("quantize", "dequantize", "gemm", "rmsnorm", "rmsnorm_backward", "gated", "gated_backward"):
        assert len(re.findall(rf"_launch\(\w+(\.device)?, lib\.mxfp4_fp8_{name},", text)) == 1, name
