"""Which stream a call of the binding runs on, without a GPU: the caller's, or the current
device's current one, with a torch that has the undocumented raw-handle call and without."""
import types

import pytest
import torch

import activation_quantized_gemm_wq_b200 as wq


@pytest.fixture
def device_three(monkeypatch):
    monkeypatch.setattr(wq, "_raw_stream", None)
    monkeypatch.setattr(wq, "_current_device", lambda: 3)


def test_current_stream_by_the_raw_handle(device_three, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    assert wq._stream(None) == 103
    assert wq._stream(None) == 103


def test_current_stream_without_the_raw_handle(device_three, monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(cuda_stream=200 + d))
    assert wq._stream(None) == 203
    assert wq._stream(None) == 203


def test_the_callers_stream():
    assert wq._stream(17) == 17
    assert wq._stream(types.SimpleNamespace(cuda_stream=18)) == 18
