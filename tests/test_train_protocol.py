"""Host models of the mbarrier protocols of the training attention kernels
(speech_encoder_b200/csrc/k_attention_train.cu), run under random schedules with
the hardware's parity rule, as test_attention_protocol.py does for the inference
kernel.  Every run checks that all actors finish, that every parity test aims at
the phase it means, and that no buffer is written or read early.

Forward: TMA into a 4-stage ring, the product warp (scores two tiles ahead into
three buffers, P V in order), four softmax warps that share nothing but the
barriers and so drift up to two tiles apart.  The negative control drops the wait
for the last but one P V before the wait for the last.

Backward: TMA into a 3-stage ring, the product warp (next scores once S has been
read, next dP once the products of dS are done), eight elementwise warps."""
import random

import pytest

from test_attention_protocol import Bar, ProtocolError


def _drive(rng, actors, tensor, tma, on_op, on_land, max_steps=400000):
    # some actors seldom get a turn: that is how warps drift apart
    weights = {k: rng.choice([0.02, 1.0, 3.0]) for k in actors}
    done = set()
    for _ in range(max_steps):
        choices = [k for k in actors if k not in done] + (["tensor"] if tensor else []) + (["tma"] if tma else [])
        if not choices:
            return
        k = rng.choices(choices, [weights.get(k, 1.0) for k in choices])[0]
        if k == "tensor":
            op = tensor.pop(0)
            if op[0] == "commit":
                op[1].arrive()
            else:
                on_op(op)
        elif k == "tma":
            what, bar = tma.pop(rng.randrange(len(tma)))
            on_land(what)
            bar.arrive()
        else:
            try:
                next(actors[k])
            except StopIteration:
                done.add(k)
    raise ProtocolError("no progress: deadlock")


def _wait(bar, phase, who):
    while not bar.test(phase & 1, phase, who):
        yield


def forward(nkv, seed, ordered_final=True, move_prob=0.2):
    rng = random.Random(seed)
    W, STAGES = 4, 4
    q_full = Bar("q_full", 1)
    kv_full, kv_empty = [[Bar(f"{n}{i}", 1) for i in range(STAGES)] for n in ("kv_full", "kv_empty")]
    s_full, p_full = [Bar(f"s_full{i}", 1) for i in range(3)], [Bar(f"p_full{i}", W) for i in range(3)]
    pv_done = [Bar(f"pv_done{i}", 1) for i in range(2)]
    tensor, tma, landed, s_ran, pv_ran, loaded, written = [], [], set(), set(), set(), {}, {}
    everyone = set(range(W))

    def producer():
        tma.append(("q", q_full))
        for j in range(nkv):
            if j >= STAGES:
                yield from _wait(kv_empty[j % STAGES], j // STAGES - 1, "producer")
                if j - STAGES not in pv_ran:
                    raise ProtocolError("stage refilled before its products ran")
            tma.append((j, kv_full[j % STAGES]))
            yield

    def product():
        def scores(j):
            yield from _wait(kv_full[j % STAGES], j // STAGES, "product kv")
            tensor.extend([("S", j), ("commit", s_full[j % 3])])

        yield from _wait(q_full, 0, "product q")
        yield from scores(0)
        if nkv > 1:
            yield from scores(1)
        for j in range(nkv):
            if j + 2 < nkv:
                if j > 0:
                    yield from _wait(pv_done[(j - 1) & 1], (j - 1) >> 1, "product pv")
                yield from scores(j + 2)
            yield from _wait(p_full[j % 3], j // 3, "product p")
            tensor.extend([("PV", j), ("commit", pv_done[j & 1]), ("commit", kv_empty[j % STAGES])])
            yield

    def softmax(w):
        for j in range(nkv):
            yield from _wait(s_full[j % 3], j // 3, f"softmax {w} S")
            loaded.setdefault(j, set()).add(w)
            yield
            if j > 0 and rng.random() < move_prob:
                yield from _wait(pv_done[(j - 1) & 1], (j - 1) >> 1, f"softmax {w} rescale")
                if j - 1 not in pv_ran or j in pv_ran:
                    raise ProtocolError("rescale races a product")
            written.setdefault(j, set()).add(w)
            p_full[j % 3].arrive()
            yield
        if ordered_final and nkv > 1:
            yield from _wait(pv_done[nkv & 1], (nkv - 2) >> 1, f"softmax {w} last but one")
        yield from _wait(pv_done[(nkv - 1) & 1], (nkv - 1) >> 1, f"softmax {w} last")
        if nkv - 1 not in pv_ran:
            raise ProtocolError("accumulator read before the last product")

    def on_op(op):
        kind, j = op
        if kind == "S":
            if j not in landed or (j >= 3 and (loaded.get(j - 3) != everyone or j - 3 not in pv_ran)):
                raise ProtocolError(f"S{j} too early")
            s_ran.add(j)
        else:
            if written.get(j) != everyone:
                raise ProtocolError(f"P{j} V before P is whole")
            pv_ran.add(j)

    actors = {"producer": producer(), "product": product(), **{f"w{w}": softmax(w) for w in range(W)}}
    _drive(rng, actors, tensor, tma, on_op, landed.add)


def backward(n, seed):
    rng = random.Random(seed)
    W, STAGES = 8, 3
    a_full, s_full, dp_full, acc_done = (Bar(k, 1) for k in ("a_full", "s_full", "dp_full", "acc_done"))
    s_read, ds_full = Bar("s_read", W), Bar("ds_full", W)
    b_full, b_empty = [[Bar(f"{k}{i}", 1) for i in range(STAGES)] for k in ("b_full", "b_empty")]
    tensor, tma, landed, ran, read_s, read_dp, written = [], [], set(), set(), {}, {}, {}
    everyone = set(range(W))

    def producer():
        tma.append(("a", a_full))
        for j in range(n):
            if j >= STAGES:
                yield from _wait(b_empty[j % STAGES], j // STAGES - 1, "producer")
                if ("acc", j - STAGES) not in ran:
                    raise ProtocolError("stage refilled before its products ran")
            tma.append((j, b_full[j % STAGES]))
            yield

    def product():
        def tile(j):
            yield from _wait(b_full[j % STAGES], j // STAGES, "product tile")

        yield from _wait(a_full, 0, "product a")
        yield from tile(0)
        tensor.extend([("S", 0), ("commit", s_full), ("dP", 0), ("commit", dp_full)])
        for j in range(n):
            if j + 1 < n:
                yield from _wait(s_read, j, "product s_read")
                yield from tile(j + 1)
                tensor.extend([("S", j + 1), ("commit", s_full)])
            yield from _wait(ds_full, j, "product ds")
            tensor.extend([("acc", j), ("commit", acc_done), ("commit", b_empty[j % STAGES])])
            if j + 1 < n:
                yield from _wait(acc_done, j, "product acc")
                tensor.extend([("dP", j + 1), ("commit", dp_full)])
            yield

    def elementwise(w):
        for j in range(n):
            yield from _wait(s_full, j, f"warp {w} S")
            read_s.setdefault(j, set()).add(w)
            s_read.arrive()
            yield
            yield from _wait(dp_full, j, f"warp {w} dP")
            read_dp.setdefault(j, set()).add(w)
            written.setdefault(j, set()).add(w)
            ds_full.arrive()
            yield
        yield from _wait(acc_done, n - 1, f"warp {w} last")
        if ("acc", n - 1) not in ran:
            raise ProtocolError("gradients read before the last product")

    def on_op(op):
        kind, j = op
        if kind in ("S", "dP") and j not in landed:
            raise ProtocolError(f"{kind}{j} before its tile")
        if kind == "S" and j > 0 and read_s.get(j - 1) != everyone:
            raise ProtocolError(f"S{j} over unread scores")
        if kind == "dP" and j > 0 and ("acc", j - 1) not in ran:
            raise ProtocolError(f"dP{j} over dS in use")
        if kind == "acc" and written.get(j) != everyone:
            raise ProtocolError(f"dS{j} used before it is whole")
        ran.add(op)

    actors = {"producer": producer(), "product": product(), **{f"w{w}": elementwise(w) for w in range(W)}}
    _drive(rng, actors, tensor, tma, on_op, landed.add)


@pytest.mark.parametrize("n", list(range(1, 10)))
def test_forward_protocol_holds_under_random_schedules(n):
    for seed in range(60):
        forward(n, seed * 7919 + n)


@pytest.mark.parametrize("n", list(range(1, 10)))
def test_backward_protocol_holds_under_random_schedules(n):
    for seed in range(40):
        backward(n, seed * 7919 + n)


def test_forward_model_catches_the_unordered_last_wait():
    caught = 0
    for n in (4, 5, 6, 7):
        for seed in range(100):
            try:
                forward(n, seed * 7919 + n, ordered_final=False)
            except ProtocolError:
                caught += 1
    assert caught > 0
