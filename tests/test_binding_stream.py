"""The stream a call takes when none is given: torch's current one, also with a
torch that lacks the short way to its address (torch replaced by stand-ins)."""
import sys
from types import SimpleNamespace

import pytest

import block_quantized_gemv_kq_amd as kq


@pytest.fixture
def torch_of(monkeypatch):
    def put(c):
        at = SimpleNamespace(device=0, streams={0: 0x100, 1: 0x200})
        cuda = SimpleNamespace(current_stream=lambda: SimpleNamespace(cuda_stream=at.streams[at.device]))
        monkeypatch.setitem(sys.modules, "torch", SimpleNamespace(cuda=cuda, _C=c(at)))
        monkeypatch.setattr(kq, "_current_stream", None)
        return at
    return put


def raw(at):
    return SimpleNamespace(_cuda_getDevice=lambda: at.device, _cuda_getCurrentRawStream=lambda d: at.streams[d])


@pytest.mark.parametrize("c", [raw, lambda at: SimpleNamespace(), lambda at: SimpleNamespace(_cuda_getDevice=lambda: at.device),
                               lambda at: SimpleNamespace(_cuda_getCurrentRawStream=lambda d: at.streams[d])])
def test_current_stream_is_asked_for_at_each_call(torch_of, c):
    at = torch_of(c)
    assert kq._stream(None) == 0x100
    at.streams[0] = 0x300
    assert kq._stream(None) == 0x300
    at.device = 1
    assert kq._stream(None) == 0x200


def test_given_streams():
    assert kq._stream(0) == 0 and kq._stream(77) == 77
    assert kq._stream(SimpleNamespace(cuda_stream=5)) == 5
