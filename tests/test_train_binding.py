"""The Python binding of the operators for training, without a GPU: which stream owns a workspace of its own, and
sizes that do not fit the library's integers."""
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


@pytest.mark.parametrize("shape", [(1, (1 << 32) + 512), (3, 1 << 31)])
def test_layernorm_rows_past_32_bits_are_refused(shape):
    """Their size would reach the library without its upper bits: 2^32 + 512 columns as 512."""
    x = torch.empty(shape, device="meta", dtype=torch.float16)
    v, s = torch.empty(shape[1], device="meta"), torch.empty(shape[0], device="meta")
    with pytest.raises(B.W2VError, match="columns") as e:
        B.w2v_op_layernorm_fwd(x, x, v, v, 1e-5, 0, s, s)
    assert e.value.code == B.W2V_ESHAPE
    with pytest.raises(B.W2VError, match="columns"):
        B.w2v_op_layernorm_bwd(x, x, v, v, s, s, 0, None, x, v, v)


@pytest.mark.parametrize("shape", [((1 << 32) + 1, 1, 64), (1, (1 << 32) + 2, 64), (1, 1, 64 << 32)])
def test_attention_sizes_past_32_bits_are_refused(shape):
    q = torch.empty(shape, device="meta", dtype=torch.float16)
    lse, err = torch.empty(shape[0], shape[2] // 64, shape[1], device="meta"), torch.empty(1, device="meta", dtype=torch.int32)
    with pytest.raises(B.W2VError, match="large") as e:
        B.w2v_op_attention_fwd(q, q, q, q, lse, err)
    assert e.value.code == B.W2V_ESHAPE
    with pytest.raises(B.W2VError, match="large"):
        B.w2v_op_attention_bwd(q, q, q, q, q, lse, q, q, q, err)
