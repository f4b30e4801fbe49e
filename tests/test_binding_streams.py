"""Which stream the binding hands to the library (no GPU): the current one's handle where none is given, with the
accessor that builds no Stream object and, in a torch without it, with the public one."""
from types import SimpleNamespace

import pytest
import torch

from video_diffusion_transformer_adaln_b200 import h3b


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=77))
    return monkeypatch


def test_without_the_accessor_the_public_stream_is_used(current):
    current.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert h3b._s(None) == 77


def test_the_accessor_is_asked_for_the_current_device(current):
    current.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    assert h3b._s(None) == 1003


def test_handles_pass_as_they_are():
    assert h3b._s(5) == 5 and h3b._s(0) == 0
