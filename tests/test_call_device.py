"""Calls are enqueued on the device of their tensors, whichever is current (no GPU needed: torch's devices and the library's
entry point are stood in for)."""
import contextlib
import ctypes
import types

import pytest
import torch

from selective_state_space_03_amd import binding, delta


@pytest.fixture
def devices(monkeypatch):
    """The current device, set to 0, and what torch.cuda.device makes of it."""
    now = types.SimpleNamespace(index=0)

    @contextlib.contextmanager
    def device(i):
        before, now.index = now.index, i
        yield
        now.index = before

    monkeypatch.setattr(binding, "_current_device", lambda: now.index)
    monkeypatch.setattr(torch.cuda, "device", device)
    return now


def _handles(monkeypatch, index, value):
    """The handle of a given stream, and of the current one by both ways to it."""
    dev = torch.device("cuda", index)
    stream = types.SimpleNamespace(cuda_stream=value)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: stream)
    monkeypatch.setattr(delta, "_raw_stream", lambda i: value)
    return [binding._stream(dev, stream), binding._stream(dev, None), delta._on(dev, None), delta._on(dev, stream)]


@pytest.mark.parametrize("value", [0, 0x1000])
@pytest.mark.parametrize("index", [0, 1])
def test_the_device_of_the_tensors(index, value, devices, monkeypatch):
    for handle in _handles(monkeypatch, index, value):
        met = []

        @ctypes.CFUNCTYPE(ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p)
        def entry(p, stream):
            met.append((devices.index, stream or 0))
            return 0

        call = binding.Call(entry, ctypes.c_int(0), handle, "out", ())
        assert call.run() == "out" and call.run() == "out"
        assert met == [(index, value)] * 2 and devices.index == 0
