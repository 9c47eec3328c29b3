"""The operators for training against float64: attention forward and backward,
LayerNorm forward and backward, gradient norm and clipping; strides, ragged
clips, what padded rows may hold, streams, captured graphs, and a run of all of
them as a fine-tuning step uses them."""
import math

import pytest
import torch

import train_reference as R
from speech_encoder_b200 import w2v as B

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _rand(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen) * std


def _triple(t3, layout):
    """Three [B, T, H*64] CUDA tensors of one layout from a [B, T, 3, H*64] CPU tensor."""
    Bn, T, _, D = t3.shape
    if layout == "fused":
        g = t3.cuda()
        return [g[:, :, i] for i in range(3)]
    if layout == "time":
        g = t3.permute(1, 0, 2, 3).contiguous().cuda()
        return [g[:, :, i].permute(1, 0, 2) for i in range(3)]
    if layout == "padded":
        g = torch.full((Bn, T + 3, 3, D + 64), 7.0, dtype=t3.dtype, device="cuda")
        g[:, :T, :, :D] = t3.cuda()
        return [g[:, :T, i, :D] for i in range(3)]
    return [t3[:, :, i].contiguous().cuda() for i in range(3)]


ATTENTION = [
    # dtype, batch, T, H, frames, layout
    (F16, 1, 1, 1, None, "dense"),
    (BF16, 3, 1, 2, [1, 0, 1], "dense"),
    (F16, 1, 2, 1, None, "fused"),
    (BF16, 1, 49, 12, None, "fused"),
    (F16, 2, 63, 2, None, "time"),
    (BF16, 1, 64, 3, None, "padded"),
    (F16, 1, 65, 1, None, "dense"),
    (F16, 2, 127, 2, [127, 126], "fused"),
    (BF16, 2, 128, 1, [64, 128], "time"),
    (F16, 4, 129, 2, [129, 1, 0, 128], "padded"),
    (BF16, 3, 200, 2, [65, 200, 63], "fused"),
    (F16, 2, 257, 2, [-5, 900], "dense"),  # clamped to 0 and T
    (F16, 1, 499, 12, None, "fused"),
    (BF16, 2, 799, 3, [799, 321], "fused"),
    (F16, 1, 1031, 2, [1030], "time"),
]


def _attention_case(dtype, Bn, T, H, frames, layout, poison=math.nan):
    gen = torch.Generator().manual_seed(T * 131 + Bn * 7 + H)
    t3 = _rand(gen, Bn, T, 3, H * 64)
    t3[:, :, 0] *= 1.5
    do = _rand(gen, Bn, T, H * 64, std=0.1)
    t3, do = t3.to(dtype), do.to(dtype)
    if frames is not None:
        for b, n in enumerate(frames):
            n = min(max(n, 0), T)
            t3[b, n:] = poison
            do[b, n:] = poison
    q, k, v = _triple(t3, layout)
    fr = None if frames is None else torch.tensor(frames, dtype=torch.int32, device="cuda")
    return t3, do, q, k, v, fr


def _run_attention(t3, do, q, k, v, fr, layout, stream=None, ws=None):
    Bn, T, D = q.shape
    err = _err()
    out = torch.full_like(q.contiguous(), math.nan)
    lse = torch.full((Bn, D // 64, T), math.nan, device="cuda")
    B.w2v_op_attention_fwd(q, k, v, out, lse, err, frames=fr, stream=stream)
    grads = _triple(torch.full(t3.shape, math.nan, dtype=t3.dtype), layout)
    dout = do.cuda()
    B.w2v_op_attention_bwd(dout, q, k, v, out, lse, *grads, err, frames=fr, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out, lse, grads


@pytest.mark.parametrize("dtype,Bn,T,H,frames,layout", ATTENTION)
def test_attention_matches_fp64(dtype, Bn, T, H, frames, layout):
    case = _attention_case(dtype, Bn, T, H, frames, layout)
    t3, do, q, k, v, fr = case
    out, lse, grads = _run_attention(*case, layout)
    want, tol, lse64 = R.attention(t3[:, :, 0], t3[:, :, 1], t3[:, :, 2], H, frames, do, out.cpu())
    R.close(out, want["out"], tol["out"], "out")
    got = lse.double().cpu()
    assert torch.equal(got == -math.inf, lse64 == -math.inf)
    live = lse64 > -math.inf
    # scores off by 2^-13 (see the reference), and lse itself rounded to fp32 (|lse| < 64)
    assert ((got - lse64)[live].abs() <= 2.0 ** -13 + 2.0 ** -18).all()
    for name, g in zip(("dq", "dk", "dv"), grads):
        R.close(g, want[name], tol[name], name)


@pytest.mark.parametrize("Bn", [33, 64, 70])
def test_attention_many_ragged_clips(Bn):
    """Up to 64 clips are ordered by length, more are taken as they come; some are empty, some equal."""
    gen = torch.Generator().manual_seed(Bn)
    frames = torch.randint(0, 300, (Bn,), generator=gen).tolist()
    frames[3] = frames[7] = 0
    frames[5] = frames[6]
    frames[1] = 300
    case = _attention_case(BF16, Bn, 300, 2, frames, "fused")
    t3, do, q, k, v, fr = case
    out, lse, grads = _run_attention(*case, "fused")
    want, tol, lse64 = R.attention(t3[:, :, 0], t3[:, :, 1], t3[:, :, 2], 2, frames, do, out.cpu())
    R.close(out, want["out"], tol["out"], "out")
    assert torch.equal(lse.cpu() == -math.inf, lse64 == -math.inf)
    for name, g in zip(("dq", "dk", "dv"), grads):
        R.close(g, want[name], tol[name], name)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_of_nothing_but_padding(dtype):
    case = _attention_case(dtype, 3, 140, 2, [0, 0, 0], "dense")
    out, lse, grads = _run_attention(*case, "dense")
    assert (out == 0).all() and (lse == -math.inf).all() and all((g == 0).all() for g in grads)


def test_attention_strides_of_single_entries_do_not_matter():
    """A clip of one frame, and a batch of one: torch may give these axes any stride."""
    gen = torch.Generator().manual_seed(8)
    q, k, v = (_rand(gen, 4, 1, 128).half().cuda() for _ in range(3))
    odd = torch.empty(4, 130, dtype=F16, device="cuda")  # row stride 130, unusable if it were used
    out, lse, err = torch.empty_like(q), torch.empty(4, 2, 1, device="cuda"), _err()
    kk = torch.as_strided(k, (4, 1, 128), (128, 77, 1))
    B.w2v_op_attention_fwd(q, kk, v, out, lse, err)
    assert torch.equal(out, v)  # one key: the output is its value
    one = torch.as_strided(q, (1, 4, 128), (13, 128, 1))
    res, l2 = torch.empty(1, 4, 128, dtype=F16, device="cuda"), torch.empty(1, 2, 4, device="cuda")
    B.w2v_op_attention_fwd(one, one, one, res, l2, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.isfinite(res).all() and odd.shape == (4, 130)


def test_attention_bindings_refuse_what_the_kernels_cannot_see():
    q = torch.zeros(2, 8, 128, dtype=F16, device="cuda")
    lse, err = torch.zeros(2, 2, 8, device="cuda"), _err()
    bad = [dict(k=q.float()), dict(v=q[:, :7]), dict(k=q.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(lse=lse.double()), dict(lse=lse[:, :, :7]), dict(err=err.float()), dict(k=q.cpu()),
           dict(frames=torch.zeros(2, device="cuda")), dict(frames=torch.zeros(3, dtype=torch.int32, device="cuda")),
           dict(q=torch.zeros(2, 8, 100, dtype=F16, device="cuda")),
           dict(v=torch.zeros(2, 8, 256, dtype=F16, device="cuda")[:, :, ::2])]
    for change in bad:
        a = dict(q=q, k=q, v=q, out=q, lse=lse, err=err)
        a.update(change)
        with pytest.raises(B.W2VError):
            B.w2v_op_attention_fwd(**a)
    with pytest.raises(B.W2VError):  # expanded over the batch: no stride to walk
        e = q[:1].expand(2, 8, 128)
        B.w2v_op_attention_fwd(e, e, e, q, lse, err)
    with pytest.raises(B.W2VError):
        w = torch.zeros(1, 300, 128, dtype=F16, device="cuda")
        B.w2v_op_attention_bwd(w, w, w, w, w, torch.zeros(1, 2, 300, device="cuda"), w, w, w, err,
                               ws=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_attention_calls_at_once_on_two_streams():
    cases = [_attention_case(F16, 2, 500, 4, [500, 210], "fused"), _attention_case(BF16, 3, 333, 4, [1, 333, 90], "dense")]
    alone = [_run_attention(*c, lay) for c, lay in zip(cases, ("fused", "dense"))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    runs = []
    for (t3, do, q, k, v, fr), s in zip(cases, streams):
        with torch.cuda.stream(s):
            err, dout = _err(), do.cuda()
            out, lse = torch.empty_like(q.contiguous()), torch.empty(q.shape[0], 4, q.shape[1], device="cuda")
            grads = [torch.empty_like(out) for _ in range(3)]
            for _ in range(5):
                B.w2v_op_attention_fwd(q, k, v, out, lse, err, frames=fr)
                B.w2v_op_attention_bwd(dout, q, k, v, out, lse, *grads, err, frames=fr)
            runs.append((out, grads, err))
    torch.cuda.synchronize()
    for (out, grads, err), one in zip(runs, alone):
        assert int(err.item()) == 0
        assert torch.equal(out, one[0]) and all(torch.equal(x, y) for x, y in zip(grads, one[2]))


def test_attention_leaves_what_lies_between_rows():
    """Rows longer than the heads' width: the columns and rows in between keep their contents."""
    dtype, Bn, T, H = F16, 2, 70, 2
    case = _attention_case(dtype, Bn, T, H, [70, 33], "padded")
    t3, do, q, k, v, fr = case
    wide = torch.full((Bn, T + 3, 3, H * 64 + 64), 7.0, dtype=dtype, device="cuda")
    grads = [wide[:, :T, i, :H * 64] for i in range(3)]
    outs = torch.full((Bn, T + 2, H * 64 + 8), 5.0, dtype=dtype, device="cuda")
    out, err = outs[:, :T, :H * 64], _err()
    dos = torch.zeros_like(outs)
    dos[:, :T, :H * 64] = do.cuda()
    lse = torch.empty(Bn, H, T, device="cuda")
    B.w2v_op_attention_fwd(q, k, v, out, lse, err, frames=fr)
    B.w2v_op_attention_bwd(dos[:, :T, :H * 64], q, k, v, out, lse, *grads, err, frames=fr)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert (outs[:, T:] == 5).all() and (outs[:, :, H * 64:] == 5).all()
    assert (wide[:, T:] == 7).all() and (wide[..., H * 64:] == 7).all()
    assert all((g[1, 33:] == 0).all() for g in (*grads, out))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,frames", [(2, None), (3, None), (5, None), (16, None), (32, None), (33, None),
                                      (64, None), (65, None), (300, [2, 32, 300, 7])])
def test_attention_gradients_of_short_sharp_clips(T, frames, dtype):
    """Rows where one key has nearly all the weight: dP - rowsum is a small difference there, which the rounding of
    out must not decide.  Each clip's gradients against the textbook's, in the Euclidean norm: an entry of dS is off by
    u |dS_ij| and by P_ij times the fp32 noise of the difference (2^-20 |dout_i| max|v_j|: sums of 64 products); that
    times |k_j| / 8 in dq_i and |q_i| / 8 in dk_j; then the result's rounding, u per entry or half the least fp16 step.
    Above 64 frames the row sum carries the rounding of out: u |dout_i| |out_i| <= u |dout_i| max|v_j|."""
    Bn, u = len(frames) if frames else 40, R.half_step(dtype)
    gen = torch.Generator().manual_seed(T)
    t3 = _rand(gen, Bn, T, 3, 64)
    t3[:, :, 0] *= 2.5
    t3, do = t3.to(dtype), _rand(gen, Bn, T, 64, std=0.05).to(dtype)
    q, k, v = _triple(t3, "fused")
    fr = None if frames is None else torch.tensor(frames, dtype=torch.int32, device="cuda")
    out, _, grads = _run_attention(t3, do, q, k, v, fr, "fused")
    for b in range(Bn):
        n = frames[b] if frames else T
        qd, kd, vd, dd = (x[b, :n].double() for x in (t3[:, :, 0], t3[:, :, 1], t3[:, :, 2], do))
        p, dp = torch.softmax(qd @ kd.T / 8, 1), dd @ vd.T
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        noise = (2.0 ** -20 + (u if n > 64 else 0)) * dd.norm(dim=1, keepdim=True) * vd.norm(dim=1).max()
        off = (u * ds.abs() + p * noise) / 8
        for name, want, got, lim in (("dq", ds @ kd / 8, grads[0], off @ kd.norm(dim=1)),
                                     ("dk", ds.T @ qd / 8, grads[1], off.T @ qd.norm(dim=1))):
            limit = 1.001 * lim.norm() + 1.01 * u * want.norm() + 2.0 ** -25 * math.sqrt(want.numel())
            error = (got[b, :n].double().cpu() - want).norm()
            assert error <= limit, (name, b, float(error), float(limit))


@pytest.mark.parametrize("poison", [math.inf, -math.inf, math.nan, 60000.0, -60000.0])
def test_attention_ignores_padded_rows(poison):
    a = _attention_case(F16, 2, 150, 2, [97, 150], "fused", poison=0.0)
    b = _attention_case(F16, 2, 150, 2, [97, 150], "fused", poison=poison)
    ra, rb = _run_attention(*a, "fused"), _run_attention(*b, "fused")
    assert torch.equal(ra[0], rb[0]) and torch.equal(ra[1], rb[1])
    assert all(torch.equal(x, y) for x, y in zip(ra[2], rb[2]))


def test_attention_repeats_bit_for_bit_whatever_the_workspace_holds():
    case = _attention_case(BF16, 2, 333, 4, [333, 120], "fused")
    n = B.w2v_op_attention_bwd_workspace(2, 333, 4)
    first = _run_attention(*case, "fused", ws=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    again = _run_attention(*case, "fused", ws=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(first[0], again[0]) and all(torch.equal(x, y) for x, y in zip(first[2], again[2]))


@pytest.mark.parametrize("exponent", [-18, -14, -6, 6, 12])
def test_attention_fp16_gradients_scale_with_dout(exponent):
    """dS is held in fp16 under a scale of its own, the row sums in pieces of their own: gradients of small and
    large dout are as exact as any (half a step of what fp16 can still say of them)."""
    case = list(_attention_case(F16, 1, 160, 2, None, "dense"))
    t3 = case[0]
    base = _run_attention(*case, "dense")
    case[1] = (case[1].float() * 2.0 ** exponent).half()
    moved = _run_attention(*case, "dense")
    want, tol, _ = R.attention(t3[:, :, 0], t3[:, :, 1], t3[:, :, 2], 2, None, case[1], moved[0].cpu())
    for name, g in zip(("dq", "dk", "dv"), moved[2]):
        R.close(g, want[name], tol[name], name)
    assert torch.equal(base[0], moved[0])


def test_attention_sharp_and_extreme_scores():
    """One key takes all the weight; scores up to +-1500: no overflow, gradients match the formula."""
    gen = torch.Generator().manual_seed(3)
    T, H = 130, 1
    t3 = _rand(gen, 1, T, 3, 64).half()
    t3[:, :, 0] = 14.0 * torch.sign(t3[:, :, 0])
    t3[:, :, 1] = 14.0 * torch.sign(t3[:, :, 1])
    t3[0, 77, 1] = t3[0, 5, 0]       # a perfect match: score 14 * 14 * 64 / 8
    do = _rand(gen, 1, T, 64).half()
    q, k, v = _triple(t3, "dense")
    out, lse, grads = _run_attention(t3, do, q, k, v, None, "dense")
    want, tol, lse64 = R.attention(t3[:, :, 0], t3[:, :, 1], t3[:, :, 2], H, None, do, out.cpu())
    # scores are multiples of 49 with magnitudes to 1568: exact in fp32 before the
    # base change, off by 2^-23 * 1568 * 1.45 (about 2^-12) after it, once more for lse
    extra = 2.0 ** -10
    assert (lse.double().cpu() - lse64).abs().max() <= extra
    for name, g in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        assert torch.isfinite(g).all()
    R.close(out, want["out"], tol["out"] * (1 + extra / R.half_step(F16)), "out")
    for name, g in zip(("dq", "dk", "dv"), grads):
        R.close(g, want[name], tol[name] * (1 + extra / R.half_step(F16)), name)


def test_attention_fp16_log_sum_exp_beyond_the_first_constant():
    """Scores of 2^21: one key takes all the weight, exactly; 8 lse needs the second group of fp16 pieces."""
    gen = torch.Generator().manual_seed(13)
    T = 140
    sign = torch.sign(_rand(gen, T, 64))
    t3 = torch.stack([512 * sign, 512 * sign, _rand(gen, T, 64)], 1)[None].half()
    do = _rand(gen, 1, T, 64).half()
    q, k, v = _triple(t3, "dense")
    out, lse, grads = _run_attention(t3, do, q, k, v, None, "dense")
    assert torch.equal(out, v) and (lse == 2.0 ** 21).all()
    assert torch.equal(grads[2].cpu(), do)
    # dP and the row sum are one number summed in two orders: 64 * 2^-23 of its magnitude, times 512 / 8
    mag = (do.double().abs() * t3[:, :, 2].double().abs()).sum(2, keepdim=True)
    for g in grads[:2]:
        assert (g.double().cpu().abs() <= 64 * 64 * 2.0 ** -23 * mag + R.tiny(F16)).all()


def test_attention_gradient_against_differences():
    """The kernel's gradients predict the change of the float64 loss along random directions."""
    case = _attention_case(F16, 1, 40, 1, None, "dense")
    t3, do, *_ = case
    out, _, grads = _run_attention(*case, "dense")
    x = [t3[0, :, i].double() for i in range(3)]

    def loss(q, k, v):
        return (torch.softmax(q @ k.T / 8, 1) @ v * do[0].double()).sum()

    gen = torch.Generator().manual_seed(9)
    for i in range(3):
        d = torch.randn(40, 64, generator=gen, dtype=torch.float64)
        h = 1e-4
        up, down = [t.clone() for t in x], [t.clone() for t in x]
        up[i] += h * d
        down[i] -= h * d
        slope = (loss(*up) - loss(*down)) / (2 * h)
        g = grads[i][0].double().cpu()
        # each entry is off by a few half steps (2^-11); 2560 of them add up in the mean square
        off = 8 * 2.0 ** -11 * float((g * d).square().sum().sqrt()) + 4 * 2.0 ** -11 * float(g.abs().max()) * 51
        assert abs(float((g * d).sum() - slope)) <= off


def test_attention_in_a_captured_graph_and_on_another_stream():
    a = _attention_case(BF16, 2, 180, 3, [180, 77], "fused")
    t3, do, q, k, v, fr = a
    expect = _run_attention(*a, "fused")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = _run_attention(*a, "fused", stream=s)
    assert torch.equal(expect[0], other[0]) and all(torch.equal(x, y) for x, y in zip(expect[2], other[2]))

    err, dout = _err(), do.cuda()
    out, lse = torch.empty_like(q.contiguous()), torch.empty(2, 3, 180, device="cuda")
    grads = [torch.empty_like(out) for _ in range(3)]
    ws = torch.empty(B.w2v_op_attention_bwd_workspace(2, 180, 3), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.w2v_op_attention_fwd(q, k, v, out, lse, err, frames=fr)
        B.w2v_op_attention_bwd(dout, q, k, v, out, lse, *grads, err, frames=fr, ws=ws)
    for n in ([180, 77], [33, 180]):  # the lengths live on the device: a replay follows them
        fr.copy_(torch.tensor(n, dtype=torch.int32))
        q[torch.isnan(q)] = 0.5
        k[torch.isnan(k)] = 0.5
        v[torch.isnan(v)] = 0.5
        dout[torch.isnan(dout)] = 0.5
        g.replay()
        eager = _run_attention(t3, dout.cpu(), q, k, v, fr, "fused")
        assert int(err.item()) == 0
        assert torch.equal(out, eager[0]) and all(torch.equal(x, y) for x, y in zip(grads, eager[2]))


def test_attention_forward_agrees_with_the_inference_kernel():
    """Both compute the same softmax of fp16 inputs; each output is two roundings from it."""
    gen = torch.Generator().manual_seed(4)
    T, H = 300, 2
    t3 = _rand(gen, 1, T, 3, H * 64).half()
    q, k, v = _triple(t3, "dense")
    t_pad = 304
    vt = torch.zeros(1, H, 64, t_pad, dtype=F16, device="cuda")
    vt[..., :T] = v.unflatten(2, (H, 64)).permute(0, 2, 3, 1)
    ref, err = torch.empty_like(q), _err()
    assert B.w2v_op_attention(q, k, vt, ref, 1, T, H, t_pad, err) == 0
    out, lse = torch.empty_like(q), torch.empty(1, H, T, device="cuda")
    B.w2v_op_attention_fwd(q, k, v, out, lse, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # the inference kernel rounds its exponents to fp16: 8 half steps of the largest value
    assert (ref.float() - out.float()).abs().max() <= 8 * 2.0 ** -11 * float(v.abs().max())


def test_attention_in_a_row_with_the_inference_kernels():
    """Kernels that start early behind one another and all want tensor memory: the inference attention (all of it),
    a GEMM, both training passes, in one queue."""
    gen = torch.Generator().manual_seed(21)
    T, H, t_pad = 700, 4, 704
    t3 = _rand(gen, 1, T, 3, H * 64).half()
    q, k, v = _triple(t3, "dense")
    vt = torch.zeros(1, H, 64, t_pad, dtype=F16, device="cuda")
    vt[..., :T] = v.unflatten(2, (H, 64)).permute(0, 2, 3, 1)
    do = _rand(gen, 1, T, H * 64, std=0.1).half().cuda()
    W = _rand(gen, H * 64, H * 64, std=0.1).half().cuda()
    err = _err()

    def queue():
        inf, out, gemm = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        lse, grads = torch.empty(1, H, T, device="cuda"), [torch.empty_like(q) for _ in range(3)]
        assert B.w2v_op_attention(q, k, vt, inf, 1, T, H, t_pad, err) == 0
        B.w2v_op_attention_fwd(q, k, v, out, lse, err)
        assert B.w2v_op_gemm(out, W, T, H * 64, H * 64, None, None, 0, gemm, 0, 0, err) == 0
        B.w2v_op_attention_bwd(do, q, k, v, out, lse, *grads, err)
        return inf, out, gemm, *grads

    runs = [queue() for _ in range(30)]
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


# ------------------------------------------------------------------ LayerNorm

LN_TYPES = [(F16, F16), (BF16, BF16), (F32, F32), (F32, F16), (F32, BF16)]
LN_SHAPES = [(1, 1), (5, 2), (3, 7), (49, 768), (33, 1024), (17, 255), (64, 512), (9, 1032), (2, 2341), (3, 8192),
             (4, 4099), (700, 40)]


def _ln_case(rows, cols, xt, yt, offset=0, pad=0):
    gen = torch.Generator().manual_seed(rows * 31 + cols)

    def make(dtype, std, shift=0.0):
        buf = torch.full((rows * (cols + pad) + offset,), 3.0, dtype=dtype, device="cuda")
        t = buf[offset:].view(rows, cols + pad)[:, :cols]
        t.copy_((_rand(gen, rows, cols, std=std) + shift).to(dtype))
        return t

    x, dy, dres = make(xt, 1.5, 0.4), make(yt, 0.2), make(xt, 0.2)
    gamma, beta = 1 + _rand(gen, cols, std=0.2), _rand(gen, cols, std=0.2)
    return x, dy, dres, gamma.cuda(), beta.cuda()


def _check_ln(rows, cols, xt, yt, act, offset=0, pad=0, residual=True):
    x, dy, dres, gamma, beta = _ln_case(rows, cols, xt, yt, offset, pad)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dgamma, dbeta = torch.full((cols,), math.nan, device="cuda"), torch.full((cols,), math.nan, device="cuda")
    B.w2v_op_layernorm_fwd(x, y, gamma, beta, 1e-5, act, mean, rstd)
    B.w2v_op_layernorm_bwd(dy, x, gamma, beta, mean, rstd, act, dres if residual else None, dx, dgamma, dbeta)
    torch.cuda.synchronize()
    c = lambda t: t.detach().cpu()  # noqa: E731
    y64, mean64, rstd64 = R.layernorm_forward(c(x), c(gamma), c(beta), 1e-5, act)
    # fp32 sums of `cols` terms, 32 to a thread and then a tree: 2^-24 * (32 + 13) of the mean magnitude
    e = 2.0 ** -18
    big = c(x).double().abs().mean(1)
    assert ((c(mean).double() - mean64).abs() <= e * big).all()
    # the variance is a sum of squares of (x - mean), whose own error is e * big against a spread 1 / rstd
    rel = e * (1 + big * rstd64)
    assert ((c(rstd).double() - rstd64).abs() <= 2 * rel * rstd64).all()
    z_mag = ((c(x).double() - mean64[:, None]).abs() * rstd64[:, None] * c(gamma).double().abs()
             + c(gamma).double().abs() + c(beta).double().abs())
    R.close(y, y64, R.half_step(yt) * y64.abs() + 4 * rel[:, None] * z_mag + R.tiny(yt), "y")
    want, mag = R.layernorm_backward(c(dy), c(x), c(gamma), c(beta), c(mean), c(rstd), act,
                                     c(dres) if residual else None)
    R.close(dx, want["dx"], R.half_step(xt) * want["dx"].abs() + 2.0 ** -18 * mag["dx"] + R.tiny(xt), "dx")
    # rows add up one after the other within a group, then over groups and blocks
    s = (2.0 ** -20 + 2.0 ** -24 * (rows / 8 + 40))
    for name, g in (("dgamma", dgamma), ("dbeta", dbeta)):
        R.close(g, want[name], s * mag[name] + 1e-30, name)


@pytest.mark.parametrize("xt,yt", LN_TYPES)
@pytest.mark.parametrize("rows,cols", LN_SHAPES)
def test_layernorm_matches_fp64(rows, cols, xt, yt):
    _check_ln(rows, cols, xt, yt, act=0)


@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("xt,yt", LN_TYPES)
def test_layernorm_gelu_matches_fp64(xt, yt, act):
    _check_ln(40, 512, xt, yt, act, residual=False)
    _check_ln(13, 77, xt, yt, act)


@pytest.mark.parametrize("xt,yt", LN_TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (8, 3)])
def test_layernorm_strides_and_alignment(xt, yt, offset, pad):
    _check_ln(11, 256, xt, yt, 0, offset, pad)


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_layernorm_affine_vectors_anywhere(shift):
    """gamma and beta inside a larger buffer, on 4-, 8- and 16-byte boundaries."""
    x, dy, dres, gamma, beta = _ln_case(100, 512, F16, F16)
    flat = torch.zeros(2, 512 + shift, device="cuda")
    g, b = flat[0, shift:], torch.empty(512 + shift, device="cuda")[shift:]
    g.copy_(gamma)
    b.copy_(beta)
    runs = []
    for gg, bb in ((gamma, beta), (g, b)):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd, dg, db = (torch.empty(n, device="cuda") for n in (100, 100, 512, 512))
        B.w2v_op_layernorm_fwd(x, y, gg, bb, 1e-5, 1, mean, rstd)
        B.w2v_op_layernorm_bwd(dy, x, gg, bb, mean, rstd, 1, dres, dx, dg, db)
        runs.append((y, dx, dg, db))
    for a, c in zip(*runs):  # sums of the unaligned path run in another order: a few roundings of fp32
        assert (a.float() - c.float()).abs().max() <= 2.0 ** -10 * c.float().abs().max()


def test_layernorm_many_rows_and_repeat():
    _check_ln(20011, 256, BF16, BF16, 1)
    x, dy, dres, gamma, beta = _ln_case(3001, 512, F16, F16)
    mean, rstd = torch.zeros(3001, device="cuda"), torch.ones(3001, device="cuda")
    runs = []
    for fill in (0, 255):
        ws = torch.full((B.w2v_op_layernorm_bwd_workspace(3001, 512),), fill, dtype=torch.uint8, device="cuda")
        dx, dg, db = torch.empty_like(x), torch.empty(512, device="cuda"), torch.empty(512, device="cuda")
        B.w2v_op_layernorm_bwd(dy, x, gamma, beta, mean, rstd, 0, None, dx, dg, db, ws=ws)
        runs.append((dx, dg, db))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_layernorm_no_rows_and_residual_in_place():
    x = torch.empty(0, 256, device="cuda")
    g, v = torch.ones(256, device="cuda"), torch.empty(0, device="cuda")
    B.w2v_op_layernorm_fwd(x, x, g, g, 1e-5, 0, v, v)
    dg, db = torch.full((256,), math.nan, device="cuda"), torch.full((256,), math.nan, device="cuda")
    B.w2v_op_layernorm_bwd(x, x, g, g, v, v, 0, None, x, dg, db)
    assert (dg == 0).all() and (db == 0).all()
    x, dy, dres, gamma, beta = _ln_case(50, 768, F32, F16)
    mean, rstd = torch.zeros(50, device="cuda"), torch.ones(50, device="cuda")
    dg, db, dx = torch.empty(768, device="cuda"), torch.empty(768, device="cuda"), torch.empty_like(x)
    B.w2v_op_layernorm_bwd(dy, x, gamma, beta, mean, rstd, 0, dres, dx, dg, db)
    B.w2v_op_layernorm_bwd(dy, x, gamma, beta, mean, rstd, 0, dres, dres, dg, db)
    assert torch.equal(dx, dres)


def test_layernorm_rows_of_infinity_stay_in_their_row():
    x, dy, dres, gamma, beta = _ln_case(20, 512, F16, F16)
    x[3] = math.inf
    x[7, 5] = math.nan
    y, mean, rstd = torch.empty_like(x), torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    B.w2v_op_layernorm_fwd(x, y, gamma, beta, 1e-5, 0, mean, rstd)
    bad = ~torch.isfinite(y).all(1)
    assert bad.nonzero().flatten().tolist() == [3, 7]


# --------------------------------------------------------------- gradient clip


def _clip_ref(grads, scale, max_norm):
    norm = scale * math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    by = min(1.0, max_norm / (norm + 1e-6)) * scale
    return norm, [g.double() * by for g in grads]


def _check_clip(grads, outs, scale, max_norm):
    before = [g.clone() for g in grads]
    norm = torch.empty(1, device="cuda")
    B.w2v_op_grad_clip(grads, outs, scale, max_norm, norm)
    want, values = _clip_ref(before, scale, max_norm)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    for i, (o, w) in enumerate(zip(outs, values)):
        # the factor is rounded to fp32, the product to the output's type
        tol = (R.half_step(o.dtype) + 2.0 ** -23) * w.abs().cpu() + R.tiny(o.dtype)
        R.close(o, w.cpu(), tol, f"tensor {i}")
    return float(norm)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_norm", [0.25, 1e9, math.inf])
def test_grad_clip_mixed_tensors(max_norm, in_place):
    gen = torch.Generator(device="cuda").manual_seed(5)
    sizes = [1, 7, 8, 1000, 8191, 8192, 8193, 0, 70001, 513 * 1025, 3]
    grads = [torch.randn(n, generator=gen, device="cuda").to((F32, F16, BF16)[i % 3]) for i, n in enumerate(sizes)]
    _check_clip(grads, grads if in_place else [torch.empty_like(g) for g in grads], 1 / 8, max_norm)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_grad_clip_any_alignment(dtype, shift):
    """Tensors packed back to back, outputs on the same and on other 16-byte offsets than their gradients."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    sizes = [5, 1, 2, 8200, 17, 30000]
    flat = torch.randn(sum(sizes) + 8, generator=gen, device="cuda").to(dtype)
    out = torch.full_like(flat, 9.0)
    grads, outs = list(flat[1:1 + sum(sizes)].split(sizes)), list(out[1 + shift:1 + shift + sum(sizes)].split(sizes))
    _check_clip(grads, outs, 1.0, 2.0)
    assert (out[:1 + shift] == 9).all() and (out[1 + shift + sum(sizes):] == 9).all()


def test_grad_clip_more_tensors_than_one_launch():
    gen = torch.Generator(device="cuda").manual_seed(7)
    grads = [torch.randn(1 + i % 37, generator=gen, device="cuda") for i in range(1300)]
    _check_clip(grads, [torch.empty_like(g) for g in grads], 0.5, 1.0)
    norm = torch.full((1,), 9.0, device="cuda")
    B.w2v_op_grad_clip([], [], 1.0, 1.0, norm)
    assert float(norm) == 0


def test_grad_clip_ranges_and_non_finite():
    big = torch.full((5000,), 1e30, device="cuda")
    small = torch.full((5000,), 1e-30, device="cuda")
    _check_clip([big], [torch.empty_like(big)], 1.0, 1.0)
    norm, out = torch.empty(1, device="cuda"), torch.empty_like(small)
    B.w2v_op_grad_clip([small], [out], 1.0, 1.0, norm)
    assert abs(float(norm) / (1e-30 * math.sqrt(5000)) - 1) < 1e-6 and torch.equal(out, small)
    for bad in (math.inf, -math.inf, math.nan):
        g = torch.ones(100, device="cuda")
        g[50] = bad
        out = torch.empty_like(g)
        B.w2v_op_grad_clip([g], [out], 0.5, 1.0, norm)
        assert not math.isfinite(float(norm))
        assert (out[:50] == 0.5).all() and (out[51:] == 0.5).all()


def test_grad_clip_binding_refuses_unlike_lists():
    a, b = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    norm = torch.empty(1, device="cuda")
    bad = [([a], [b, b]), ([a], [b.half()]), ([a], [b[:7]]), ([torch.ones(4, 4, device="cuda").t()], [torch.ones(4, 4, device="cuda")]),
           ([a, b.half()], [torch.ones(8, device="cuda").half(), torch.ones(8, device="cuda")]), ([a], [b.cpu()]), ([a, a], [a, b])]
    for grads, outs in bad:
        with pytest.raises(B.W2VError):
            B.w2v_op_grad_clip(grads, outs, 1.0, 1.0, norm)


def test_grad_clip_in_a_captured_graph():
    g = torch.ones(20000, device="cuda")
    out, norm = torch.empty_like(g), torch.empty(1, device="cuda")
    ws = torch.empty(B.w2v_op_grad_clip_workspace(1), dtype=torch.uint8, device="cuda")
    B.w2v_op_grad_clip([g], [out], 1.0, 1.0, norm, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.w2v_op_grad_clip([g], [out], 1.0, 1.0, norm, ws=ws)
    for value in (2.0, 1e-4):
        g.fill_(value)
        graph.replay()
        want, _ = _clip_ref([g], 1.0, 1.0)
        assert abs(float(norm) - want) <= 1e-6 * want


# -------------------------------------------------- a block's step, as it is used


def test_attention_sublayer_step():
    """y = x + attention(LN(x) Wqkv) of a pre-norm block on a padded batch: the gradients of the operators, chained
    as a training step chains them, against autograd in float64; then all of them clipped."""
    gen = torch.Generator().manual_seed(11)
    Bn, T, H = 3, 75, 4
    d, frames = 64 * H, [75, 40, 1]
    x = _rand(gen, Bn * T, d)
    W = _rand(gen, 3 * d, d, std=1 / math.sqrt(d))
    gamma, beta = 1 + _rand(gen, d, std=0.1), _rand(gen, d, std=0.1)
    gy = _rand(gen, Bn, T, d, std=0.1)
    for b, n in enumerate(frames):
        gy[b, n:] = 0

    xg, Wg, gg, bg, gyg = (t.cuda() for t in (x, W, gamma, beta, gy))
    fr, err = torch.tensor(frames, dtype=torch.int32, device="cuda"), _err()
    n1, mean, rstd = torch.empty(Bn * T, d, dtype=F16, device="cuda"), *(torch.empty(Bn * T, device="cuda") for _ in "ab")
    B.w2v_op_layernorm_fwd(xg, n1, gg, bg, 1e-5, 0, mean, rstd)
    Wh = Wg.half()
    qkv = (n1 @ Wh.T).view(Bn, T, 3, d)
    out, lse = torch.empty(Bn, T, d, dtype=F16, device="cuda"), torch.empty(Bn, H, T, device="cuda")
    B.w2v_op_attention_fwd(qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], out, lse, err, frames=fr)
    dqkv = torch.empty_like(qkv)
    B.w2v_op_attention_bwd(gyg.half(), qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], out, lse, dqkv[:, :, 0],
                           dqkv[:, :, 1], dqkv[:, :, 2], err, frames=fr)
    dflat = dqkv.view(Bn * T, 3 * d)
    dW, dn1 = dflat.T @ n1, dflat @ Wh
    dx, dgamma, dbeta = torch.empty_like(xg), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    B.w2v_op_layernorm_bwd(dn1, xg, gg, bg, mean, rstd, 0, gyg.view(Bn * T, d), dx, dgamma, dbeta)

    leaves = [t.double().requires_grad_(True) for t in (x, W, gamma, beta)]
    xd, Wd, gd, bd = leaves
    z = (xd - xd.mean(1, keepdim=True)) / torch.sqrt(xd.var(1, unbiased=False, keepdim=True) + 1e-5) * gd + bd
    p3 = (z @ Wd.T).view(Bn, T, 3, H, 64)
    loss = (xd.view(Bn, T, d) * gy.double()).sum()
    for b, n in enumerate(frames):
        q, k, v = (p3[b, :n, i].transpose(0, 1) for i in range(3))
        o = torch.softmax(q @ k.transpose(1, 2) / 8, -1) @ v
        loss = loss + (o.transpose(0, 1).reshape(n, d) * gy[b, :n].double()).sum()
    want = torch.autograd.grad(loss, leaves)
    assert int(err.item()) == 0
    # Eight fp16 roundings lie between the leaves and each gradient (LN, W, qkv, P,
    # out, dS, dqkv, dn1), each 2^-11 relative to its tensor: their root sum of
    # squares is 3 * 2^-11 of a gradient's norm at most; the bound is four times that.
    for name, got, ref in zip(("dx", "dW", "dgamma", "dbeta"), (dx, dW, dgamma, dbeta), want):
        ref = ref.view(got.shape)
        off = float((got.double().cpu() - ref).norm() / ref.norm())
        assert off <= 12 * 2.0 ** -11, (name, off)

    grads = [dx.clone(), dW, dgamma, dbeta]
    _check_clip(grads, grads, 1.0, 0.5)
