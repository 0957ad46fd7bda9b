"""Which streams the binding lets a beam selection run on (no GPU: devices and streams are stand-ins)."""
import types

import pytest
import torch

import device_draft_verification_amd as sv
from device_draft_verification_amd import binding


class Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)
        self.cuda_stream = 0x1000 + index


class Library:
    """Takes the calls that the binding lets through."""

    def __init__(self):
        self.calls = []

    def _call(self, name):
        def f(*args):
            self.calls.append(name)
            return 0
        return f

    def __getattr__(self, name):
        return self._call(name)


@pytest.fixture
def two_devices(monkeypatch):
    lib, at = Library(), types.SimpleNamespace(device=0)
    monkeypatch.setattr(binding, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at.device)
    monkeypatch.setattr(binding, "_current_stream", lambda device: 0x2000 + device)
    return lib, at


def test_a_context_takes_streams_of_its_own_device_only(two_devices):
    lib, at = two_devices
    with pytest.raises(ValueError, match="spec_beam_init.*cuda:1"):
        sv.spec_beam_init(1, 2, 2, 100, torch.float32, stream=Stream(1))
    assert lib.calls == []
    ctx = sv.spec_beam_init(1, 2, 2, 100, torch.float32, stream=Stream(0))
    sv.spec_beam_set_stream(ctx, Stream(0))
    sv.spec_beam_set_stream(ctx)
    assert lib.calls == ["spec_beam_init"] + ["spec_beam_set_stream"] * 2
    with pytest.raises(ValueError, match="spec_beam_set_stream.*cuda:1"):
        sv.spec_beam_set_stream(ctx, Stream(1))
    at.device = 1                       # the current stream is another device's
    with pytest.raises(ValueError, match="current device is cuda:1"):
        sv.spec_beam_set_stream(ctx)
    sv.spec_beam_set_stream(ctx, Stream(0))
    assert lib.calls.count("spec_beam_set_stream") == 3
    sv.spec_beam_init(1, 2, 2, 100, torch.float32, stream=Stream(1))
    with pytest.raises(ValueError, match="spec_beam_init"):
        sv.spec_beam_init(1, 2, 2, 100, torch.float32, stream=Stream(0))
