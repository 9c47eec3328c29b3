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


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("T", [1, 2, 20, 64, 70, 140])
def test_attention_shows_values_that_are_not_finite(T, which, value, dtype):
    """One channel of one live row of q, k or v, at every index modulo 8 and in every tile."""
    for at in sorted({j for j in (*range(8), 63, 64, 65, 127, 128, T - 1) if j < T}):
        t3, do = _one_head(dtype, T, 5)
        t3[at, which, 9] = value
        _check_pattern(t3, do)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_attention_shows_them_beside_padded_rows(value, dtype):
    for frames, at in ((1, 0), (2, 1), (66, 64), (66, 3), (130, 129)):
        t3, do = _one_head(dtype, 150, 6)
        t3[frames:], do[frames:] = math.nan, math.nan
        t3[at, 1, 0] = value
        _check_pattern(t3, do, frames)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 2, 9, 100])
def test_attention_rows_without_a_score(T, dtype):
    """Every score of a row is -infinity: no softmax."""
    t3, do = _one_head(dtype, T, 7)
    t3[0, 0, 3] = -math.inf
    t3[:, 1, 3] = 1.0
    _check_pattern(t3, do)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_scores_of_minus_infinity_before_others(dtype):
    """The first tile's scores are all -infinity, the second's are not: the row has the second's softmax."""
    t3, do = _one_head(dtype, 100, 8)
    t3[:, 0, 3] = 1.0
    t3[:70, 1, 3] = -math.inf
    _check_pattern(t3, do)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("at", range(8))
def test_attention_overflowed_scores(at, sign):
    """A product of finite rows that passes fp32's range: +infinity, which shows, or -infinity, a weight of zero."""
    t3, do = _one_head(BF16, 40, 9)
    t3[:, :2, 2] = 0.0
    t3[1, 0, 2], t3[at, 1, 2] = 1e30, sign * 1e10
    got, lse = _kernels(t3, do)
    bad = torch.zeros(40, dtype=torch.bool)
    bad[1] = sign > 0
    assert torch.equal(torch.isnan(lse), bad)
    for name, rows in (("out", bad), ("dq", bad), ("dk", bad.any().expand(40)), ("dv", bad.any().expand(40))):
        assert torch.equal(~torch.isfinite(got[name]), rows[:, None].expand(40, 64)), name


# --------------------------------------------------------- streams given by handle


def _owner(address):
    """The stream whose pool holds an address of torch's allocator."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not an address of the allocator")


def test_workspaces_belong_to_the_default_stream_when_it_is_named():
    dev = torch.device("cuda", torch.cuda.current_device())
    side = torch.cuda.Stream()
    for stream, handle in ((None, 0), (0, 0), (torch.cuda.default_stream(), 0), (side, side.cuda_stream),
                           (side.cuda_stream, side.cuda_stream)):
        pointer, _, owner = B._workspace(None, 1 << 12, dev, stream)
        assert pointer == owner.data_ptr() and _owner(pointer) == handle
    with torch.cuda.stream(side):  # the default stream by name, from another one
        pointer, _, owner = B._workspace(None, 1 << 12, dev, 0)
        assert _owner(pointer) == 0


@pytest.mark.parametrize("by", ["handle", "object"])
def test_calls_on_the_default_stream_by_name(by):
    """With other streams allocating and writing meanwhile, the results are those of the same calls unnamed."""
    stream = 0 if by == "handle" else torch.cuda.default_stream()
    gen = torch.Generator().manual_seed(12)
    q, k, v, do = (torch.randn(2, 500, 256, generator=gen).half().cuda() for _ in range(4))
    x, gamma = torch.randn(6000, 512, generator=gen).cuda(), torch.ones(512, device="cuda")
    err, sides = _err(), [torch.cuda.Stream() for _ in range(8)]

    def calls(s):
        out, lse = torch.empty_like(q), torch.empty(2, 4, 500, device="cuda")
        grads = [torch.empty_like(q) for _ in range(3)]
        dx, mean, rstd = torch.empty_like(x), torch.zeros(6000, device="cuda"), torch.ones(6000, device="cuda")
        dg, db, norm = (torch.empty(n, device="cuda") for n in (512, 512, 1))
        B.w2v_op_attention_fwd(q, k, v, out, lse, err, stream=s)
        B.w2v_op_attention_bwd(do, q, k, v, out, lse, *grads, err, stream=s)
        B.w2v_op_layernorm_bwd(x, x, gamma, gamma, mean, rstd, 0, None, dx, dg, db, stream=s)
        B.w2v_op_grad_clip([dx], [dx], 1.0, 1.0, norm, stream=s)
        return (*grads, dx, dg, db, norm)

    alone = calls(None)
    torch.cuda.synchronize()
    for _ in range(10):
        got = calls(stream)
        for s in sides:
            with torch.cuda.stream(s):
                torch.full((1 << 18,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(alone, got))


# ------------------------------------------------------ memory shared row by row


def test_layernorm_operands_between_one_another():
    """fp32 rows, their fp16 rows and the gradients side by side in the rows of one buffer: apart, though their
    ranges are not."""
    gen = torch.Generator().manual_seed(14)
    rows, cols = 90, 256
    wide = torch.zeros(rows, 4 * cols, device="cuda")
    x, dx, dres, half = (wide[:, i * cols:(i + 1) * cols] for i in range(4))
    half = half.view(F16)
    y, dy = half[:, :cols], half[:, cols:]
    x.copy_(torch.randn(rows, cols, generator=gen))
    dres.copy_(torch.randn(rows, cols, generator=gen))
    dy.copy_(torch.randn(rows, cols, generator=gen))
    gamma, beta = torch.randn(2, cols, generator=gen).cuda()
    stats = torch.empty(2, rows, device="cuda")
    sums = torch.empty(4, cols, device="cuda")
    B.w2v_op_layernorm_fwd(x, y, gamma, beta, 1e-5, 1, *stats)
    B.w2v_op_layernorm_bwd(dy, x, gamma, beta, *stats, 1, dres, dx, sums[0], sums[1])
    y2, dx2 = torch.empty(rows, cols, dtype=F16, device="cuda"), torch.empty(rows, cols, device="cuda")
    stats2 = torch.empty(2, rows, device="cuda")
    B.w2v_op_layernorm_fwd(x.contiguous(), y2, gamma, beta, 1e-5, 1, *stats2)
    B.w2v_op_layernorm_bwd(dy.contiguous(), x.contiguous(), gamma, beta, *stats2, 1, dres.contiguous(), dx2, sums[2],
                           sums[3])
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(stats, stats2) and torch.equal(sums[:2], sums[2:])
    with pytest.raises(B.W2VError):
        B.w2v_op_layernorm_bwd(dy, x, gamma, beta, *stats, 1, dres, x, sums[0], sums[1])
    with pytest.raises(B.W2VError):
        B.w2v_op_layernorm_fwd(x, wide[:, 1:cols + 1], gamma, beta, 1e-5, 0, *stats)


def test_attention_gradients_over_their_operands_are_refused():
    q, k, v, do = torch.randn(4, 2, 70, 128, device="cuda").half()
    out, lse, err = torch.empty_like(q), torch.empty(2, 2, 70, device="cuda"), _err()
    B.w2v_op_attention_fwd(q, k, v, out, lse, err)
    dq, dk, dv = torch.empty(3, 2, 70, 128, dtype=F16, device="cuda")
    B.w2v_op_attention_bwd(do, q, k, v, out, lse, dq, dk, dv, err)
    for bad in ((q, dk, dv), (dq, k, dv), (dq, dk, do), (dq, dq, dv), (out, dk, dv)):
        with pytest.raises(B.W2VError):
            B.w2v_op_attention_bwd(do, q, k, v, out, lse, *bad, err)
    with pytest.raises(B.W2VError):
        B.w2v_op_attention_fwd(q, k, v, v, lse, err)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("frames", [None, [300, 0, 129, 128, 64, 1]])
def test_attention_output_over_its_queries(frames, dtype):
    """Without a backward pass to come, out may take the place of q (here, in a fused projection's rows)."""
    gen = torch.Generator().manual_seed(16)
    qkv = torch.randn(6, 300, 3, 192, generator=gen).to(dtype).cuda()
    fr = None if frames is None else torch.tensor(frames, dtype=torch.int32, device="cuda")
    out, err = torch.empty(6, 300, 3, 192, dtype=dtype, device="cuda")[:, :, 0], _err()
    lse, again = torch.empty(2, 6, 3, 300, device="cuda")
    q, k, v = (qkv[:, :, i] for i in range(3))
    B.w2v_op_attention_fwd(q, k, v, out, lse, err, frames=fr)
    kept = qkv[:, :, 1:].clone()
    B.w2v_op_attention_fwd(q, k, v, q, again, err, frames=fr)
    assert torch.equal(q, out) and torch.equal(lse, again) and torch.equal(qkv[:, :, 1:], kept)
    assert int(err.item()) == 0
    for args in ((q, q, v), (q, k, q)):  # as keys or values it is read by every row
        with pytest.raises(B.W2VError):
            B.w2v_op_attention_fwd(*args, q, lse, err)


# ------------------------------------------------------- GELU over its whole range


def _through_layernorm(z, xt, yt, act):
    """(f(z), f'(z)): one row with gamma 0, beta z and dy 1 has y = f(z) and dbeta = f'(z)."""
    n = len(z)
    x = torch.linspace(-1, 1, n, device="cuda").to(xt)[None]
    zero, y, dx = torch.zeros(n, device="cuda"), torch.empty(1, n, dtype=yt, device="cuda"), torch.empty_like(x)
    mean, rstd, dgamma, dbeta = (torch.empty(k, device="cuda") for k in (1, 1, n, n))
    B.w2v_op_layernorm_fwd(x, y, zero, z, 1e-5, act, mean, rstd)
    B.w2v_op_layernorm_bwd(torch.ones_like(y), x, zero, z, mean, rstd, act, None, dx, dgamma, dbeta)
    return y[0].double().cpu(), dbeta.double().cpu()


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("n", [1024, 8192, 1021, 5003])
def test_exact_gelu_over_its_range(n, xt, yt):
    """Phi(-|z|) = e g(t), e = exp(-z^2 / 2), t = 1 / (1 + p |z|), counted in u = 2^-24 of its value: t is off by 3 u
    (a rounding, and a unit of the approximate reciprocal), which g takes up to 2.6 times; e by 2.8 u (the approximate
    exponential's 2^-22.5) and 1.5 z^2 u of its argument's roundings; the polynomial by 12 u of its coefficients' and
    steps' roundings (the magnitudes of its terms are at most 1.8 times their sum) and 1.1 u of its own error; two
    products.  Together 28 u + 1.5 z^2 u, held to 2^-19 + z^2 2^-23.  With 16-bit results the polynomial's own error is
    up to 6.4e-5 of Phi(-|z|) and 6.4e-8; the value is then rounded to its type."""
    u = 2.0 ** -24
    for part in range(4):
        z = torch.linspace(-13, 13, 4 * n)[part::4].contiguous().cuda()
        y, slope = _through_layernorm(z, xt, yt, 1)
        zd = z.double().cpu()
        tail = torch.special.erfc(zd.abs() / math.sqrt(2)) / 2
        phi = torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
        relative = 2.0 ** -19 + zd * zd * 2.0 ** -23

        def off(wide):  # of Phi(-|z|)
            return tail * relative + (0 if wide else torch.minimum(6.5e-5 * tail, torch.tensor(6.5e-8)))

        cdf = torch.where(zd < 0, tail, 1 - tail)
        want = zd * cdf
        half = torch.finfo(yt).eps / 2
        limit = (half + u) * want.abs() + zd.abs() * off(yt == F32) * (1 + half) + R.tiny(yt)
        assert ((y - want).abs() <= limit).all(), float(((y - want).abs() / limit).max())
        # Phi(z) + z phi(z): two roundings of at most 1.13, and z phi with the error of e
        limit = off(xt == F32) + zd.abs() * phi * relative + 2 * 1.13 * u
        err = (slope - (cdf + zd * phi)).abs()
        assert (err <= limit).all(), float((err / limit).max())


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F16, F16)])
def test_tanh_gelu_over_its_range(xt, yt):
    """s = sigmoid(2 u(z)) with an exponent up to 2 u(13) = 172: off by 4 of its roundings and those of the approximate
    instructions, in proportion to the smaller of s and 1 - s and otherwise 2 u of s.  Below 2^-126 s counts as zero."""
    u, n = 2.0 ** -24, 4099
    z = torch.linspace(-13, 13, n).cuda()
    y, slope = _through_layernorm(z, xt, yt, 2)
    zd = z.double().cpu()
    w = 2 * math.sqrt(2 / math.pi) * (zd + 0.044715 * zd ** 3)
    s, dw = torch.sigmoid(w), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * zd * zd)
    off = s * ((4 * w.abs() + 4) * torch.sigmoid(-w) + 4) * u
    half = torch.finfo(yt).eps / 2
    want = zd * s
    limit = (half + 2 * u) * want.abs() + zd.abs() * (off + 2.0 ** -126) * (1 + half) + R.tiny(yt)
    assert ((y - want).abs() <= limit).all(), float(((y - want).abs() / limit).max())
    # s + z s (1 - s) dw: the product z s - z s s loses what it cancels, a rounding of z s times dw
    limit = (off + 2.0 ** -126) * (1 + 2 * zd.abs() * dw) + 4 * u * (s + zd.abs() * s * dw)
    err = (slope - (s + zd * s * (1 - s) * dw)).abs()
    assert (err <= limit).all(), float((err / limit).max())


# -------------------------------------------------- sums that one row more decides


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("xt,yt", [(F16, F16), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", [(1, 256), (63, 512), (64, 1024), (65, 256), (9, 2048), (300, 2048), (1184, 1024),
                                       (1185, 768), (2367, 512), (2369, 512), (7105, 256), (20011, 256), (4737, 255),
                                       (301, 1027)])
def test_layernorm_affine_gradients_count_every_row_once(rows, cols, xt, yt, residual):
    """Small whole numbers with mean 0 and rstd 1: every partial sum is a whole number below 2^24, so dgamma and dbeta
    are exact, and a row left out, or taken twice, shows."""
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randint(-4, 5, (rows, cols), generator=gen, device="cuda")
    dy = torch.randint(-8, 9, (rows, cols), generator=gen, device="cuda")
    dy[:, 0], x[:, 0] = 3, 1  # a column that counts them
    one, zero = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    dgamma, dbeta = torch.full((2, cols), math.nan, device="cuda")
    xx, res = x.to(xt), torch.zeros(rows, cols, dtype=xt, device="cuda")
    B.w2v_op_layernorm_bwd(dy.to(yt), xx, one, zero, torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"), 0,
                           res if residual else None, torch.empty_like(xx), dgamma, dbeta)
    assert torch.equal(dgamma.long(), (dy * x).sum(0)) and torch.equal(dbeta.long(), dy.sum(0))
    assert int(dbeta[0]) == int(dgamma[0]) == 3 * rows


# --------------------------------------------- short clips, many of them, some empty


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("Bn,T", [(3, 100), (33, 100), (64, 128), (70, 100), (70, 17)])
def test_attention_many_short_ragged_clips(Bn, T, dtype):
    """Up to 128 frames one launch makes the statistics, the gradients and the zeros of empty clips; up to 64 clips it
    takes them by length, more as they come."""
    gen = torch.Generator().manual_seed(Bn * T)
    frames = torch.randint(0, T + 1, (Bn,), generator=gen).tolist()
    frames[0], frames[1], frames[-1] = 0, T, 0
    t3 = torch.randn(Bn, T, 3, 128, generator=gen).to(dtype)
    do = (0.1 * torch.randn(Bn, T, 128, generator=gen)).to(dtype)
    for b, n in enumerate(frames):
        t3[b, n:], do[b, n:] = math.nan, math.nan
    q, k, v = (t3.cuda()[:, :, i] for i in range(3))
    out, lse, err = torch.full((Bn, T, 128), math.nan, dtype=dtype, device="cuda"), torch.empty(Bn, 2, T, device="cuda"), _err()
    grads = [torch.full_like(out, math.nan) for _ in range(3)]
    fr = torch.tensor(frames, dtype=torch.int32, device="cuda")
    B.w2v_op_attention_fwd(q, k, v, out, lse, err, frames=fr)
    B.w2v_op_attention_bwd(do.cuda(), q, k, v, out, lse, *grads, err, frames=fr)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want, tol, lse64 = R.attention(t3[:, :, 0], t3[:, :, 1], t3[:, :, 2], 2, frames, do, out.cpu())
    R.close(out, want["out"], tol["out"], "out")
    assert torch.equal(lse.cpu() == -math.inf, lse64 == -math.inf)
    for name, g in zip(("dq", "dk", "dv"), grads):
        R.close(g, want[name], tol[name], name)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [5, 100, 300])
def test_attention_of_empty_clips_alone(T, dtype):
    q = torch.full((3, T, 64), math.nan, dtype=dtype, device="cuda")
    out, lse, err = q.clone(), torch.zeros(3, 1, T, device="cuda"), _err()
    grads, fr = [q.clone() for _ in range(3)], torch.tensor([0, -3, 0], dtype=torch.int32, device="cuda")
    B.w2v_op_attention_fwd(q, q, q, out, lse, err, frames=fr)
    B.w2v_op_attention_bwd(q, q, q, q, out, lse, *grads, err, frames=fr)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and (lse == -math.inf).all() and all((t == 0).all() for t in (out, *grads))


@pytest.mark.parametrize("rows,cols,xt,yt", [(40, 513, F32, F16), (300, 2048, F16, F16), (3000, 255, BF16, BF16),
                                             (2400, 512, F32, F32)])
def test_layernorm_residual_in_place_at_other_widths(rows, cols, xt, yt):
    gen = torch.Generator().manual_seed(cols)
    x, dres = (torch.randn(rows, cols, generator=gen).to(xt).cuda() for _ in range(2))
    dy = torch.randn(rows, cols, generator=gen).to(yt).cuda()
    gamma, beta = torch.randn(2, cols, generator=gen).cuda()
    mean, rstd, y = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(dy)
    B.w2v_op_layernorm_fwd(x, y, gamma, beta, 1e-5, 2, mean, rstd)
    dx, sums = torch.empty_like(x), torch.empty(4, cols, device="cuda")
    B.w2v_op_layernorm_bwd(dy, x, gamma, beta, mean, rstd, 2, dres, dx, sums[0], sums[1])
    B.w2v_op_layernorm_bwd(dy, x, gamma, beta, mean, rstd, 2, dres, dres, sums[2], sums[3])
    assert torch.equal(dx, dres) and torch.equal(sums[:2], sums[2:])


# --------------------------------------------------------------- gradient norm


@pytest.mark.parametrize("scale,max_norm", [(2.0 ** -20, 1.0), (1.0, 0.1), (2.0 ** -10, 2.0 ** -30), (2.0 ** -140, math.inf)])
def test_grad_clip_factors_below_fp32(scale, max_norm):
    """Large gradients take factors that fp32 holds only as subnormals: the products are as exact as any (three
    roundings: the factor's, and those of the product)."""
    gen = torch.Generator().manual_seed(15)
    g = torch.cat([torch.full((100,), 1e37), 1e37 * torch.randn(900, generator=gen)]).cuda()
    small = torch.randn(50, generator=gen).cuda()  # ends below fp32's range
    outs, norm = [torch.empty_like(g), torch.empty_like(small)], torch.empty(1, device="cuda")
    B.w2v_op_grad_clip([g, small], outs, scale, max_norm, norm)
    want = scale * math.sqrt(math.fsum(float(t.double().square().sum()) for t in (g, small)))
    by = min(1.0, max_norm / (want + 1e-6)) * scale
    assert abs(float(norm) - want) <= 2.0 ** -23 * want + R.tiny(F32)
    for o, t in zip(outs, (g, small)):
        R.close(o, t.double().cpu() * by, 3 * 2.0 ** -24 * t.double().cpu().abs() * by + 2 * R.tiny(F32), "out")


def test_grad_clip_norm_past_fp32():
    """A norm that fp64 holds and fp32 does not is written as infinity, and clips nothing, as any infinite one."""
    g = torch.full((5000,), 3e38, device="cuda")
    out, norm = torch.empty_like(g), torch.empty(1, device="cuda")
    B.w2v_op_grad_clip([g], [out], 0.5, 1.0, norm)
    assert float(norm) == math.inf and torch.equal(out, g * 0.5)
    B.w2v_op_grad_clip([g], [out], 2.0 ** -20, 1.0, norm)  # 2e34 after unscaling: clipped again
    want = 3e38 * 2.0 ** -20 * math.sqrt(5000)
    assert abs(float(norm) / want - 1) < 1e-6 and abs(float(out[7]) * math.sqrt(5000) - 1) < 1e-6
