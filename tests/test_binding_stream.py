"""The stream a binding call goes to when none is named: the current one, by the short way and by the public one."""
import pytest
import torch

from quantized_verification_gb300 import qv


class FakeStream:
    cuda_stream = 0x5150


def test_public_way_where_the_short_one_is_missing(monkeypatch):
    monkeypatch.setattr(qv, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", FakeStream)
    assert qv._stream(None) == FakeStream.cuda_stream
    assert qv._stream(77) == 77


def test_short_way_asks_for_the_current_device(monkeypatch):
    monkeypatch.setattr(qv, "_device", lambda: 3)
    monkeypatch.setattr(qv, "_raw_stream", lambda device: 1000 + device)
    assert qv._stream(None) == 1003


def test_pointers_of_what_is_no_tensor_are_refused():
    assert qv._ptr(None) is None
    for what in (3, b"bytes", [1.0], torch.UntypedStorage(4)):
        with pytest.raises((TypeError, ValueError)):
            qv._ptr(what)


@pytest.mark.gpu
def test_both_ways_agree(monkeypatch):
    from gpu_util import require_gpu
    require_gpu()
    side = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(stream):
            short = qv._stream(None)
            with monkeypatch.context() as m:
                m.setattr(qv, "_raw_stream", None)
                assert qv._stream(None) == short == stream.cuda_stream
