"""The operators for training at the edges of their inputs: values that are not
finite, streams given by handle, memory that overlaps, GELU over its whole range,
and sums that a single row decides."""
import math

import pytest
import torch

import train_reference as R
from speech_encoder_b200 import w2v as B

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------- attention: values that are not finite


def _dot(a, b):
    """a b^T with every product formed (a library product may leave out a factor of zero)."""
    return (a[:, None, :] * b[None, :, :]).sum(-1)


def _definition(q, k, v, do):
    """out, lse and the gradients of one head, float64, from the formulas."""
    s = _dot(q, k) / 8
    p = torch.softmax(s, 1)
    out, dp = _dot(p, v.T), _dot(do, v)
    ds = p * (dp - (p * dp).sum(1, keepdim=True))
    return dict(out=out, lse=torch.log(torch.exp(s).sum(1)), dq=_dot(ds, k.T) / 8, dk=_dot(ds.T, q.T) / 8,
                dv=_dot(p.T, do.T)), p


def _one_head(dtype, T, seed):
    gen = torch.Generator().manual_seed(seed)
    t3 = torch.randn(T, 3, 64, generator=gen).to(dtype)
    return t3, (0.1 * torch.randn(T, 64, generator=gen)).to(dtype)


def _kernels(t3, do, frames=None):
    q, k, v = (t3[None, :, i].contiguous().cuda() for i in range(3))
    out, lse, err = torch.zeros_like(q), torch.zeros(1, 1, len(t3), device="cuda"), _err()
    grads = [torch.zeros_like(q) for _ in range(3)]
    fr = None if frames is None else torch.tensor([frames], dtype=torch.int32, device="cuda")
    B.w2v_op_attention_fwd(q, k, v, out, lse, err, frames=fr)
    B.w2v_op_attention_bwd(do[None].cuda(), q, k, v, out, lse, *grads, err, frames=fr)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return {n: t[0].double().cpu() for n, t in zip(("out", "dq", "dk", "dv"), (out, *grads))}, lse[0, 0].double().cpu()


def _check_pattern(t3, do, frames=None):
    n = len(t3) if frames is None else frames
    want, p = _definition(*(t3[:n, i].double() for i in range(3)), do[:n].double())
    got, lse = _kernels(t3, do, frames)
    for name in ("out", "dq", "dk", "dv"):
        assert torch.equal(torch.isfinite(got[name][:n]), torch.isfinite(want[name])), name
        assert (got[name][n:] == 0).all()
    assert torch.equal(torch.isfinite(lse[:n]), torch.isfinite(want["lse"]))
    # rows that are finite keep their values: roundings as in the reference's tolerances
    u = R.half_step(t3.dtype)
    tol = u * want["out"].abs() + (u + R.FP32_SLACK) * _dot(p, t3[:n, 2].double().abs().T) + R.tiny(t3.dtype)
    ok = torch.isfinite(want["out"])
    assert ((got["out"][:n] - want["out"]).abs() <= tol)[ok].all()
    good = torch.isfinite(want["lse"])
    assert ((lse[:n] - want["lse"]).abs() <= 2.0 ** -13 + 2.0 ** -18)[good].all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [2, 20, 64, 70, 100, 140])
def test_attention_key_at_minus_infinity(T, dtype):
    """A live key that every row's score is -infinity for has a weight of zero: nothing of it reaches out, dv or the
    finite channels of dq (0 * infinity is left in its own), whatever columns the last tile has past the clip."""
    for at in sorted({0, 1, 5 % T, T - 1}):
        t3, do = _one_head(dtype, T, 4)
        t3[:, 0, 3], t3[at, 1, 3] = 1.0, -math.inf
        _check_pattern(t3, do)
