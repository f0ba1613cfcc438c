"""The stream handle that the binding passes on, without a GPU: torch's calls are replaced."""
import types

import pytest

from top_group_sparse_gb300 import qsa


def test_the_current_stream_with_and_without_torchs_private_call(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    assert qsa._stream(None) == 1003
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert qsa._stream(None) == 77


def test_streams_that_are_given():
    assert qsa._stream(5) == 5 and qsa._stream(0) == 0
    assert qsa._stream(types.SimpleNamespace(cuda_stream=9)) == 9
