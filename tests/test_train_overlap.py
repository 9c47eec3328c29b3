"""Operands of the training calls that share memory: refused by every call (no GPU
needed, no pointer is read), and told exactly from operands that lie between one
another's rows (csrc/extent.h, compiled here, against sets of bytes)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from speech_encoder_b200 import w2v as B
from test_train_refusals import P, _clip, _shape

CSRC = os.path.join(os.path.dirname(B.__file__), "csrc")
MB = 1 << 20
FWD = ("q", "k", "v", "out", "lse", "err")
BWD = ("dout", "q", "k", "v", "out", "lse", "dq", "dk", "dv", "ws", "err")


def _apart(names):
    return {n: P + 16 * MB * i for i, n in enumerate(names)}


def _fwd(s, a):
    return B.lib().w2v_op_attention_fwd(ctypes.byref(s), *(a[n] for n in FWD), None)


def _bwd(s, a):
    return B.lib().w2v_op_attention_bwd(ctypes.byref(s), *(a[n] for n in BWD[:10]), 1 << 24, a["err"], None)


@pytest.mark.parametrize("T", [10, 200])
def test_attention_outputs_over_other_operands(T):
    s = _shape(T=T, qkv_bs=256 * T, out_bs=256 * T, grad_bs=256 * T)
    last = 2 * (2 * T - 1) * 256  # the last row's first byte
    for out in ("out", "lse", "err"):
        for other in set(FWD) - {out}:
            a = _apart(FWD)
            for at in (a[other], a[other] + (last if other in ("q", "k", "v", "out") else 0)):
                if (out, other, at) == ("out", "q", a["q"]):
                    continue  # in place: allowed
                assert _fwd(s, dict(a, **{out: at})) == B.W2V_EINVAL, (out, other)
    for out in ("dq", "dk", "dv", "err") + (("ws",) if T > 128 else ()):
        for other in set(BWD) - {out} - (set() if T > 128 else {"ws"}):
            a = _apart(BWD)
            assert _bwd(s, dict(a, **{out: a[other]})) == B.W2V_EINVAL, (out, other)


def test_attention_rows_that_meet_between_rows():
    """Three operands of one fused buffer lie apart; one moved by a row's 8 elements meets its neighbour."""
    s = _shape(qkv_ld=768, qkv_bs=7680, grad_ld=768, grad_bs=7680)
    a = _apart(BWD)
    a.update(dq=P + 900 * MB, dk=P + 900 * MB + 512, dv=P + 900 * MB + 1024 - 16)
    assert _bwd(s, a) == B.W2V_EINVAL
    frames = _shape(frames=P + 16 * MB * FWD.index("out") + 64)
    assert _fwd(frames, _apart(FWD)) == B.W2V_EINVAL


def _ln(forward, **kw):
    rows, cols = 300, 64
    names = ("x", "y", "gamma", "beta", "mean", "rstd") if forward else (
        "dy", "x", "gamma", "beta", "mean", "rstd", "dres", "dx", "dgamma", "dbeta", "ws")
    a = dict(_apart(names), **{k: v for k, v in kw.items() if k in names})
    ld = kw.get("ld", cols)
    L = B.lib()
    if forward:
        return L.w2v_op_layernorm_fwd(a["x"], 2, ld, a["y"], 2, ld, rows, cols, a["gamma"], a["beta"], 1e-5, 0,
                                      a["mean"], a["rstd"], None)
    return L.w2v_op_layernorm_bwd(a["dy"], 2, ld, a["x"], 2, ld, rows, cols, a["gamma"], a["beta"], a["mean"], a["rstd"],
                                  0, a["dres"], ld, a["dx"], ld, a["dgamma"], a["dbeta"], a["ws"], 1 << 24, None)


def test_layernorm_outputs_over_other_operands():
    names = ("x", "y", "gamma", "beta", "mean", "rstd")
    for out in ("y", "mean", "rstd"):
        for other in set(names) - {out}:
            assert _ln(True, **{out: _apart(names)[other]}) == B.W2V_EINVAL, (out, other)
    names = ("dy", "x", "gamma", "beta", "mean", "rstd", "dres", "dx", "dgamma", "dbeta", "ws")
    for out in ("dx", "dgamma", "dbeta", "ws"):
        for other in set(names) - {out}:
            if {out, other} != {"dx", "dres"}:
                assert _ln(False, **{out: _apart(names)[other]}) == B.W2V_EINVAL, (out, other)
    # the sum in place is one address and one stride, nothing beside it
    assert _ln(False, dx=_apart(names)["dres"] + 256) == B.W2V_EINVAL
    # rows of a wider buffer: gamma within one of y's rows
    assert _ln(True, ld=128, gamma=_apart(("x", "y"))["y"] + 3 * 512 + 252) == B.W2V_EINVAL


def test_grad_clip_norm_and_workspace_over_tensors():
    n = B.w2v_op_grad_clip_workspace(1)
    g, o, ws, norm = P, P + MB, P + 2 * MB, P + 3 * MB
    for norm_at in (g, g + 28, o + 28, ws, ws + n - 4):
        assert _clip(grads=(g,), outs=(o,), norm=norm_at, ws=ws) == B.W2V_EINVAL
    for ws_at in (g, o, g + 32 - n, o + 16, norm - 16):
        assert _clip(grads=(g,), outs=(o,), norm=norm, ws=ws_at) == B.W2V_EINVAL


SHIM = """
#include "extent.h"
extern "C" int meet(const int64_t* v) {  // at, width, stride0, n0, stride1, n1, twice; -1: refused
  w2v::Extent e[2];
  for (int i = 0; i < 2; ++i, v += 6)
    if (!w2v::make_extent(reinterpret_cast<const void*>(v[0]), v[1], v[2], v[3], v[4], v[5], &e[i])) return -1;
  return w2v::overlap(e[0], e[1]);
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("extent")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-shared", "-fPIC", "-I",
                    CSRC, str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    f = ctypes.CDLL(str(d / "shim.so")).meet

    def call(a, b):
        return f((ctypes.c_int64 * 12)(*a, *b))
    return call


def _bytes(at, width, s0, n0, s1, n1):
    return {at + i * s0 + k * s1 + w for i in range(n0) for k in range(n1) for w in range(width)}


def _draw(rng, width):
    """An operand whose strides nest, as the calls have them: rows apart, whichever stride is the longer."""
    n0, n1 = rng.choice([0, 1, 2, 3, 5]), rng.choice([1, 1, 2, 4])
    if rng.random() < 0.3:  # time-major: the second stride is the shorter one
        outer = width + rng.choice([0, 4])
        inner = outer * n1 + rng.choice([0, 2, 24])
    else:
        inner = width + rng.choice([0, 0, 1, 3, 8, 16])
        outer = inner * max(n0, 1) + rng.choice([0, 0, 2, 8])
    return [rng.randrange(1000, 1060), width, inner, n0, outer, n1]


def test_overlap_against_sets_of_bytes(meet):
    rng = random.Random(3)
    seen = [0, 0]
    for _ in range(30000):
        a = _draw(rng, rng.choice([1, 2, 4, 8]))
        b = _draw(rng, rng.choice([1, 2, 4, 8]))
        if rng.random() < 0.5:  # slices of one buffer
            b[2:] = a[2:]
            b[1] = min(b[1], a[1])
        want = bool(_bytes(*a) & _bytes(*b))
        seen[want] += 1
        assert meet(a, b) == want and meet(b, a) == want, (a, b)
    assert min(seen) > 3000


def test_overlap_at_full_size(meet):
    """The slices of a fused projection, and rows of unlike operands in one buffer, at sizes past 32 bits."""
    T, n, w = 1 << 20, 64, 2048
    q, k, v = ([1 << 40, w, 3 * w, T, 3 * w * T, n], [(1 << 40) + w, w, 3 * w, T, 3 * w * T, n],
               [(1 << 40) + 2 * w, w, 3 * w, T, 3 * w * T, n])
    assert not meet(q, k) and not meet(q, v) and not meet(k, v) and meet(q, q)
    v[0] += 16  # its rows reach into the next row of q
    assert not meet(k, v) and meet(q, v)
    # the last row alone
    assert meet(q, [(1 << 40) + 3 * w * (T * n - 1) + w - 16, 16, 0, 1, 0, 1])
    assert not meet(q, [(1 << 40) + 3 * w * (T * n - 1) + w, 16, 0, 1, 0, 1])
    # longer than any memory
    assert meet([1 << 20, 8, 1 << 50, 1 << 20, 0, 1], q) == -1
