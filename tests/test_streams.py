"""The stream that a call without one runs on."""
import types

import pytest
import torch

import rank_fp8_residual_b200 as ll


@pytest.fixture
def fake_cuda(monkeypatch):
    now = types.SimpleNamespace(device=1, streams={0: 70, 1: 71})
    monkeypatch.setattr(ll, "_current_stream", None, raising=False)
    monkeypatch.setattr(ll, "_raw_stream", None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now.device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(cuda_stream=now.streams[now.device if d is None else d]))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now.device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now.streams[d], raising=False)
    return now


@pytest.mark.parametrize("missing", [(), ("_cuda_getDevice",), ("_cuda_getCurrentRawStream",),
                                     ("_cuda_getDevice", "_cuda_getCurrentRawStream")])
def test_current_stream_of_the_current_device(fake_cuda, monkeypatch, missing):
    """With and without torch's functions for the handle alone."""
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    for device, stream in ((1, 71), (0, 70), (0, 72)):
        fake_cuda.device, fake_cuda.streams[device] = device, stream
        assert ll._stream(None) == stream


def test_a_function_of_another_meaning_is_not_used(fake_cuda, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 5)
    assert ll._stream(None) == 71
    monkeypatch.setattr(ll, "_current_stream", None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda: 71)
    assert ll._stream(None) == 71


def test_given_streams():
    assert ll._stream(0) == 0 and ll._stream(17) == 17
    assert ll._stream(types.SimpleNamespace(cuda_stream=19)) == 19
