"""The stream a call goes to by default (no GPU): torch's current one, asked for the short way where torch has it."""
import types

import pytest

import moe_expert_load_ultraep_amd as U

torch = pytest.importorskip("torch")


def test_given_streams_are_taken():
    assert U._stream(77) == 77
    assert U._stream(types.SimpleNamespace(cuda_stream=78)) == 78


@pytest.mark.parametrize("short", [True, False])
def test_current_stream(monkeypatch, short):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=79))
    if short:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 80 + device, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert U._stream(None) == (83 if short else 79)
