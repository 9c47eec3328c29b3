"""Argument checks of the operators for training (no GPU needed: every refusal
comes before anything is launched, and no pointer is read)."""
import ctypes
import math

import pytest
import torch

from speech_encoder_b200 import w2v as B

P = 1 << 20  # an aligned address that no call may read


def _shape(**kw):
    f = dict(dtype=0, batch=2, T=10, H=4, qkv_ld=256, qkv_bs=2560, out_ld=256, out_bs=2560, grad_ld=256, grad_bs=2560,
             frames=None)
    f.update(kw)
    return B.w2v_attention_shape(*[f[n] for n, _ in B.w2v_attention_shape._fields_])


def _fwd(s, **kw):
    a = dict(q=P, k=P, v=P, out=P, lse=P, err=P)
    a.update(kw)
    return B.lib().w2v_op_attention_fwd(None if s is None else ctypes.byref(s), *a.values(), None)


def _bwd(s, ws_bytes=1 << 30, **kw):
    a = dict(dout=P, q=P, k=P, v=P, out=P, lse=P, dq=P, dk=P, dv=P, ws=P)
    a.update(kw)
    return B.lib().w2v_op_attention_bwd(ctypes.byref(s), *a.values(), ws_bytes, P, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), B.W2V_EINVAL), (dict(dtype=-1), B.W2V_EINVAL), (dict(batch=0), B.W2V_ESHAPE),
    (dict(T=0), B.W2V_ESHAPE), (dict(T=-1), B.W2V_ESHAPE), (dict(H=0), B.W2V_ESHAPE), (dict(T=1 << 24), B.W2V_ESHAPE),
    (dict(batch=1 << 20, H=1 << 20), B.W2V_ESHAPE),
    (dict(T=(1 << 24) - 1, batch=1 << 12, H=16), B.W2V_ESHAPE),
    (dict(qkv_ld=248), B.W2V_EINVAL), (dict(qkv_ld=260), B.W2V_EINVAL), (dict(qkv_bs=2564), B.W2V_EINVAL),
    (dict(qkv_bs=0), B.W2V_EINVAL), (dict(qkv_bs=512), B.W2V_EINVAL), (dict(qkv_ld=-256), B.W2V_EINVAL),
    (dict(out_ld=255), B.W2V_EINVAL), (dict(out_bs=256), B.W2V_EINVAL), (dict(qkv_ld=1 << 39), B.W2V_EINVAL)])
def test_attention_shape_refused(change, code):
    assert _fwd(_shape(**change)) == code
    assert _bwd(_shape(**change)) == code


def test_attention_gradient_strides_refused():
    assert _bwd(_shape(grad_ld=192)) == B.W2V_EINVAL
    assert _bwd(_shape(grad_bs=8)) == B.W2V_EINVAL


@pytest.mark.parametrize("bad", [None, P + 8])
def test_attention_pointers_refused(bad):
    s = _shape()
    for name in ("q", "k", "v", "out"):
        assert _fwd(s, **{name: bad}) == B.W2V_EINVAL, name
    for name in ("dout", "q", "k", "v", "out", "dq", "dk", "dv"):
        assert _bwd(s, **{name: bad}) == B.W2V_EINVAL, name
    assert _fwd(s, lse=None) == B.W2V_EINVAL
    assert _fwd(s, lse=P + 2) == B.W2V_EINVAL
    assert _fwd(s, err=None) == B.W2V_EINVAL
    assert _fwd(s, err=P + 1) == B.W2V_EINVAL
    assert _fwd(_shape(frames=P + 2)) == B.W2V_EINVAL
    assert _fwd(None) == B.W2V_EINVAL


def test_attention_workspace():
    n = B.w2v_op_attention_bwd_workspace(2, 200, 4)
    assert n > 0
    s = _shape(T=200, qkv_bs=51200, out_bs=51200, grad_bs=51200)
    assert _bwd(s, ws_bytes=n - 1) == B.W2V_EINVAL
    for ws in (None, P + 8):
        assert _bwd(s, ws=ws) == B.W2V_EINVAL
    assert B.w2v_op_attention_bwd_workspace(2, 128, 4) == 0
    assert B.w2v_op_attention_bwd_workspace(0, 10, 4) == 0
    assert B.w2v_op_attention_bwd_workspace(2, 0, 4) == 0
    # sizes past 32 bits are counted in 64
    assert B.w2v_op_attention_bwd_workspace(64, 1 << 20, 16) > 1 << 32


def _ln_fwd(**kw):
    a = dict(x=P, x_type=0, x_ld=64, y=P, y_type=0, y_ld=64, rows=3, cols=64, gamma=P, beta=P, eps=1e-5, act=0, mean=P,
             rstd=P)
    a.update(kw)
    return B.lib().w2v_op_layernorm_fwd(*a.values(), None)


def _ln_bwd(ws_bytes=1 << 30, **kw):
    a = dict(dy=P, y_type=0, dy_ld=64, x=P, x_type=0, x_ld=64, rows=3, cols=64, gamma=P, beta=P, mean=P, rstd=P, act=0,
             dres=None, dres_ld=64, dx=P, dx_ld=64, dgamma=P, dbeta=P, ws=P)
    a.update(kw)
    return B.lib().w2v_op_layernorm_bwd(*a.values(), ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(x_type=3), B.W2V_EINVAL), (dict(y_type=1), B.W2V_EINVAL), (dict(y_type=2), B.W2V_EINVAL),
    (dict(act=3), B.W2V_EINVAL), (dict(act=-1), B.W2V_EINVAL), (dict(rows=-1), B.W2V_ESHAPE),
    (dict(rows=1 << 31), B.W2V_ESHAPE), (dict(cols=0), B.W2V_ESHAPE), (dict(cols=8193), B.W2V_ESHAPE),
    (dict(x_ld=63), B.W2V_EINVAL), (dict(x=None), B.W2V_EINVAL), (dict(x=P + 1), B.W2V_EINVAL),
    (dict(gamma=None), B.W2V_EINVAL), (dict(beta=P + 2), B.W2V_EINVAL), (dict(mean=None), B.W2V_EINVAL),
    (dict(rstd=P + 1), B.W2V_EINVAL)])
def test_layernorm_refused(change, code):
    assert _ln_fwd(**change) == code
    assert _ln_bwd(**change) == code


def test_layernorm_one_sided_refusals():
    assert _ln_fwd(eps=0.0) == B.W2V_EINVAL
    assert _ln_fwd(eps=math.nan) == B.W2V_EINVAL
    assert _ln_fwd(y_ld=10) == B.W2V_EINVAL
    for change in (dict(dx_ld=10), dict(dy_ld=10), dict(dres=P, dres_ld=10), dict(dx=None), dict(dgamma=None),
                   dict(dbeta=P + 1), dict(rows=5000, ws=None), dict(rows=5000, ws=P + 4), dict(dres=P, dres_ld=128)):
        assert _ln_bwd(**change) == B.W2V_EINVAL, change
    n = B.w2v_op_layernorm_bwd_workspace(5000, 64)
    assert n > 0 and _ln_bwd(rows=5000, ws_bytes=n - 1) == B.W2V_EINVAL
    assert B.w2v_op_layernorm_bwd_workspace(3, 64) == 0
    assert B.w2v_op_layernorm_bwd_workspace(-1, 64) == 0
    assert B.w2v_op_layernorm_bwd_workspace(3, 8193) == 0


def _clip(grads=(P,), outs=(P,), counts=(8,), types=(2,), n=None, scale=1.0, max_norm=1.0, norm=P, ws=P,
          ws_bytes=1 << 30):
    n = len(grads) if n is None else n
    m = len(grads)
    return B.lib().w2v_op_grad_clip(n, (ctypes.c_void_p * m)(*grads), (ctypes.c_void_p * m)(*outs),
                                    (ctypes.c_int64 * m)(*counts), (ctypes.c_int * m)(*types), scale, max_norm, norm,
                                    ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), B.W2V_ESHAPE), (dict(counts=(-1,)), B.W2V_ESHAPE), (dict(counts=(1 << 33,)), B.W2V_ESHAPE),
    (dict(types=(3,)), B.W2V_EINVAL), (dict(grads=(None,)), B.W2V_EINVAL), (dict(outs=(None,)), B.W2V_EINVAL),
    (dict(grads=(P + 2,), outs=(P + 2,)), B.W2V_EINVAL), (dict(scale=0.0), B.W2V_EINVAL),
    (dict(scale=math.inf), B.W2V_EINVAL), (dict(scale=math.nan), B.W2V_EINVAL), (dict(max_norm=0.0), B.W2V_EINVAL),
    (dict(max_norm=math.nan), B.W2V_EINVAL), (dict(norm=None), B.W2V_EINVAL), (dict(ws=None), B.W2V_EINVAL),
    (dict(ws=P + 8), B.W2V_EINVAL), (dict(ws_bytes=0), B.W2V_EINVAL),
    # the same tensor twice, an output over another gradient, a shifted output
    (dict(grads=(P, P), outs=(P, P), counts=(8, 8), types=(2, 2)), B.W2V_EINVAL),
    (dict(grads=(P, P + 64), outs=(P + 64, P), counts=(8, 8), types=(2, 2)), B.W2V_EINVAL),
    (dict(grads=(P,), outs=(P + 4,)), B.W2V_EINVAL),
    (dict(grads=(P, P + 16), outs=(P + 512, P + 1024), counts=(8, 8), types=(2, 2)), B.W2V_EINVAL)])
def test_grad_clip_refused(kw, code):
    assert _clip(**kw) == code


def test_bindings_refuse_tensors_off_the_gpu():
    x = torch.zeros(2, 5, 128, dtype=torch.float16)
    lse, err = torch.zeros(2, 2, 5), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(B.W2VError) as e:
        B.w2v_op_attention_fwd(x, x, x, x, lse, err)
    assert e.value.code == B.W2V_EINVAL
    r = torch.zeros(3, 64)
    with pytest.raises(B.W2VError):
        B.w2v_op_layernorm_fwd(r, r, r[0], r[0], 1e-5, 0, r[:, 0].contiguous(), r[:, 0].contiguous())
    with pytest.raises(B.W2VError):
        B.w2v_op_grad_clip([r], [r], 1.0, 1.0, torch.zeros(1))
