"""The stream that calls are made on, found with and without torch's undocumented shortcut."""
import importlib.util
import types

import torch

from decode_gemv_sign_gb300 import wcomp


def test_given_streams():
    assert wcomp._stream(7) == 7
    assert wcomp._stream(types.SimpleNamespace(cuda_stream=9)) == 9


def test_current_stream_without_the_shortcut(monkeypatch):
    """A torch that lacks it has its documented call made instead."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=11))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    spec = importlib.util.spec_from_file_location("wcomp_again", wcomp.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._stream() == 11
