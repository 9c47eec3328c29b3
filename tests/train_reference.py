"""Plain float64 forms of the operators for training, with the error that each
output may carry.

Tolerances count roundings.  u is half a step of the 16-bit type relative to the
value (fp16 2^-11, bf16 2^-8).  An output is rounded once (u |value|), and each
probability or dS entry that goes into a product is rounded once (u times the sum
of the magnitudes of the product's terms).  The rest is fp32: a score is a sum of
64 products whose magnitudes add up to at most 16 in these tests (after the 1/8),
so with a truncating accumulator it is off by at most 64 * 2^-23 * 16 = 2^-13,
which is the relative error of its probability; dP and the row sums add
64 * 2^-23 of their magnitudes.  FP32_SLACK = 2^-12 of the sums of magnitudes
covers both.
"""
import math

import torch

FP32_SLACK = 2.0 ** -12


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest subnormal: what rounding may lose next to zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def attention(q, k, v, H, frames=None, dout=None, out_saved=None):
    """(value, tolerance) of out, lse and, with dout, of dq, dk, dv; [B, T, H*64] CPU tensors.
    out_saved: the forward's rounded out, which the backward's row sums use."""
    dtype = q.dtype
    u, eps0 = half_step(dtype), tiny(dtype)
    B, T, D = q.shape
    frames = [T] * B if frames is None else list(frames)
    res = {n: torch.zeros(B, T, D, dtype=torch.float64) for n in ("out", "dq", "dk", "dv")}
    tol = {n: torch.zeros(B, T, D, dtype=torch.float64) for n in res}
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64)
    for b in range(B):
        n = min(max(frames[b], 0), T)
        if n == 0:
            continue
        for h in range(H):
            at = (b, slice(0, n), slice(64 * h, 64 * h + 64))
            qd, kd, vd = q[at].double(), k[at].double(), v[at].double()
            s = qd @ kd.T / 8
            lse[b, h, :n] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            o = p @ vd
            res["out"][at] = o
            tol["out"][at] = u * o.abs() + (u + FP32_SLACK) * (p @ vd.abs()) + eps0
            if dout is None:
                continue
            do, os = dout[at].double(), out_saved[at].double()
            dv = p.T @ do
            dp = do @ vd.T
            # clips of one tile: the row sum goes by the probabilities, not by the rounded out
            rows = ((p * dp) if n <= 64 else (do * os)).sum(1, keepdim=True)
            ds = p * (dp - rows)
            mag = p * (do.abs() @ vd.abs().T + (do * os).abs().sum(1, keepdim=True))
            if n == 1:
                ds = torch.zeros_like(ds)
            # dq has what a row of the rounded dS sums to taken out again, in proportion to P: it goes by the exact
            # row sum, and each rounding counts once with its key and once, at most, with the mean of the keys
            exact = p * (dp - (p * dp).sum(1, keepdim=True)) if n > 1 else ds
            dq, dk = exact @ kd / 8, ds.T @ qd / 8
            res["dv"][at], res["dq"][at], res["dk"][at] = dv, dq, dk
            tol["dv"][at] = u * dv.abs() + (u + FP32_SLACK) * (p.T @ do.abs()) + eps0
            each = u * ds.abs() + FP32_SLACK * mag
            mean = p @ kd.abs()
            left = each.sum(1, keepdim=True) + (do * os).abs().sum(1, keepdim=True) * u
            tol["dq"][at] = (u * dq.abs() + (each @ kd.abs() + each.sum(1, keepdim=True) * mean
                                             + 2 * u * left * mean) / 8 + eps0)
            tol["dk"][at] = u * dk.abs() + each.T @ qd.abs() / 8 + eps0
    return res, tol, lse


def close(got, want, tol, what):
    got = got.detach().double().cpu()
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = ((got - want).abs() - tol)
    assert off.max() <= 0, f"{what}: off by {(got - want).abs().max():.3e}, over the tolerance by {off.max():.3e}"


def gelu(z, act):
    """GELU in float64 (0 none, 1 exact, 2 tanh form), by autograd-friendly operations."""
    if act == 0:
        return z
    if act == 1:
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def layernorm_forward(x, gamma, beta, eps, act):
    xd = x.double()
    mean = xd.mean(1)
    rstd = 1 / torch.sqrt((xd - mean[:, None]).square().mean(1) + eps)
    z = (xd - mean[:, None]) * rstd[:, None] * gamma.double() + beta.double()
    return gelu(z, act), mean, rstd


def layernorm_backward(dy, x, gamma, beta, mean, rstd, act, dres=None):
    """The documented formulas; returns values and the magnitudes that their sums are made of."""
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    z = (xh * gamma.double() + beta.double()).requires_grad_(True)
    y = gelu(z, act)
    slope, = torch.autograd.grad(y.sum(), z)
    dz = dy.double() * slope
    w = dz * gamma.double()
    r = rstd.double()[:, None]
    m1, m2 = w.mean(1, keepdim=True), (w * xh).mean(1, keepdim=True)
    dx = r * (w - m1 - xh * m2)
    # GELU's slope is known to 2^-20 of dy (|slope| < 1.13): counted with dy itself
    base = dy.double().abs() * gamma.double().abs()
    mag = r * (base + base.mean(1, keepdim=True) + xh.abs() * (base * xh.abs()).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        mag = mag + dres.double().abs()
    return dict(dx=dx, dgamma=(dz * xh).sum(0), dbeta=dz.sum(0)), dict(
        dx=mag, dgamma=(dy.double().abs() * xh.abs()).sum(0), dbeta=dy.double().abs().sum(0))
