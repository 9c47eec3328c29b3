"""The Python binding of the operators for training, without a GPU: which stream owns a workspace of its own."""
import contextlib

import pytest
import torch

from speech_encoder_b200 import w2v as B


class _Stream:
    def __init__(self, cuda_stream, kind):
        self.cuda_stream, self.kind = cuda_stream, kind


@pytest.mark.parametrize("stream,kind", [(0, "default"), (_Stream(0, "user"), "default"), (0x7000, "external"),
                                         (_Stream(0x7000, "user"), "external")])
def test_workspace_belongs_to_the_stream_of_the_call(monkeypatch, stream, kind):
    """Handle 0 is the default stream.  torch takes an external stream of 0 for one that was not given and hands out
    one of its pool, whose memory other work may get while the call still runs."""
    entered = []

    def external(handle, device=None):
        assert handle != 0
        return _Stream(handle, "external")

    @contextlib.contextmanager
    def enter(s):
        entered.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0, "default"))
    monkeypatch.setattr(torch.cuda, "stream", enter)
    pointer, nbytes, owner = B._workspace(None, 256, torch.device("cpu"), stream)
    assert pointer == owner.data_ptr() and nbytes == 256
    assert [(s.kind, s.cuda_stream) for s in entered] == [(kind, B._stream(stream))]
