"""Host-side checks of the binding's device handling (no GPU): calls launch on the current device, so tensors of
another one are refused before anything reaches the library."""
import importlib.util

import pytest
import torch

from kda_recurrent_state_gb300 import binding


class OnDevice:
    """Stands for a CUDA tensor of device 1."""
    device = torch.device("cuda:1")

    def get_device(self):
        return 1


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="x is on cuda:1.*current device.*cuda:0"):
        binding._on_gpu(OnDevice(), "x")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert binding._on_gpu(OnDevice(), "x") == 1


def test_streams_of_another_device_are_refused(monkeypatch):
    class Stream:
        cuda_stream = 5

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream)
    with pytest.raises(ValueError, match="cuda:1.*current device.*cuda:0"):
        binding._stream(torch.device("cuda:1"))
    for device in (torch.device("cuda:0"), torch.device("cuda"), None):
        assert binding._stream(device).value == 5


def test_stream_handle_without_the_raw_accessor(monkeypatch):
    """Where torch lacks the accessor of the bare handle, the handle comes from the Stream object."""
    class Stream:
        def __init__(self, device):
            self.cuda_stream = 40 + device

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    spec = importlib.util.spec_from_file_location("binding_without_accessor", binding.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module._raw_stream(2) == 42
