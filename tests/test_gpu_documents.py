"""Head norms with rotary positions, the cross entropy of hidden states and AdamW over many tensors on the GPU, against
the oracle in 64 bits (oracle/documents_ref.py, whose bounds come from the roundings)."""
import math

import pytest
import torch

from oracle import documents_ref as R
from step_gpt_train_gb300 import gpt2 as g

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def seed():
    torch.manual_seed(11)
    torch.cuda.set_device(0)


def rnd(*shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, device="cuda") * std).to(dtype)


def near(got, want, bound, what):
    """|got - want| <= bound + half a step of got's type, where the steps of subnormals do not count."""
    far = (got.double() - want).abs() - bound - R.HALF[got.dtype] * (want.abs() + bound)
    assert torch.isfinite(got).all(), what
    assert (far <= 0).all(), f"{what}: {far.max().item():.3g} beyond the bound at {far.argmax().item()} of {far.numel()}"


def captured(run):
    """What run writes, from a replayed graph."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    return graph


# ---------------------------------------------------------------- norms and rotation

def rotary_state(dtype, rows, hq, hk, hd, rot, norm, fused, **kw):
    s = {"turns": g.gpt2_rotary_turns(rot, **kw).cuda()}
    if fused:  # queries, keys and values in one buffer, the values between guards
        s["buf"] = rnd(rows, (hq + 2 * hk) * hd, dtype=dtype)
        s["q"] = s["buf"][:, :hq * hd].unflatten(1, (hq, hd))
        s["k"] = s["buf"][:, hq * hd:(hq + hk) * hd].unflatten(1, (hk, hd))
    else:
        s["q"], s["k"] = rnd(rows, hq, hd, dtype=dtype), rnd(rows, hk, hd, dtype=dtype)
    s["q_gamma"], s["k_gamma"] = (((1 + 0.2 * rnd(hd)).to(dtype)) if norm else None for _ in range(2))
    s["eps"] = 1e-5 if norm else None
    s["pos"] = torch.randint(0, 5000, (rows,), device="cuda").int()
    return s


SHAPES = [(1, 1, 1, 64, 64), (3, 12, 12, 64, 64), (67, 16, 4, 64, 32), (129, 25, 25, 64, 16), (10, 5, 1, 64, 0),
          (33, 3, 2, 32, 32), (31, 6, 2, 16, 8), (65, 7, 7, 8, 8), (9, 4, 2, 128, 128), (8, 2, 1, 128, 48),
          (2000, 8, 2, 64, 64), (17, 4, 0, 64, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rotary(dtype, interleaved, norm, shape):
    rows, hq, hk, hd, rot = shape
    fused = rows % 2 == 1 and hk > 0
    s = rotary_state(dtype, *shape, norm, fused)
    kw = dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=s["eps"], interleaved=interleaved, amplitude=1.25)
    qo, ko = torch.empty_like(s["q"]).contiguous(), torch.empty_like(s["k"]).contiguous()
    g.gpt2_op_qk_norm_rotary_forward(qo, ko, s["q"], s["k"], s["pos"], s["turns"], **kw)
    gamma = lambda n: s[n].double() if norm else None  # noqa: E731
    for name, out in (("q", qo), ("k", ko)):
        y, bound = R.rotary(s[name].double(), s["pos"], s["turns"], gamma(name + "_gamma"), s["eps"], interleaved, 1.25)
        near(out, y, bound, name)
    # the gradients
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    dq, dk = torch.empty_like(qo), torch.empty_like(ko)
    dg = dict(dq_gamma=torch.full((hd,), 7.0, device="cuda"), dk_gamma=torch.full((hd,), 7.0, device="cuda")) if norm else {}
    run = lambda a, b: g.gpt2_op_qk_norm_rotary_backward(a, b, dqo, dko, s["q"], s["k"], s["pos"], s["turns"], **dg, **kw)  # noqa: E731
    run(dq, dk)
    for name, dy, out in (("q", dqo, dq), ("k", dko, dk)):
        dx, dgamma, bound, gbound = R.rotary_backward(dy.double(), s[name].double(), s["pos"], s["turns"],
                                                      gamma(name + "_gamma"), s["eps"], interleaved, 1.25)
        near(out, dx, bound, "d" + name)
        if norm:
            near(dg[f"d{name}_gamma"], dgamma, gbound, f"d{name}_gamma")
    # into column blocks of one buffer and in place: the same bits, nothing else touched
    if fused:
        before = s["buf"].clone()
        g.gpt2_op_qk_norm_rotary_forward(s["q"], s["k"], s["q"], s["k"], s["pos"], s["turns"], **kw)
        assert torch.equal(s["q"], qo) and torch.equal(s["k"], ko)
        assert torch.equal(s["buf"][:, (hq + hk) * hd:], before[:, (hq + hk) * hd:])
        s["buf"].copy_(before)
        run(dqo, dko)
        assert torch.equal(dqo, dq) and torch.equal(dko, dk)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_far_positions(interleaved):
    s = rotary_state(F32, 8, 2, 1, 64, 64, False, False, scaling="parts", factor=32.0, context=4096)
    s["pos"] = torch.tensor([0, 1, -1, 131071, 1 << 24, (1 << 31) - 1, -(1 << 31), 12345]).int().cuda()
    qo, ko = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    g.gpt2_op_qk_norm_rotary_forward(qo, ko, s["q"], s["k"], s["pos"], s["turns"], interleaved=interleaved)
    for name, out in (("q", qo), ("k", ko)):
        near(out, *R.rotary(s[name].double(), s["pos"], s["turns"], interleaved=interleaved), name)


def test_rotary_row_of_zeros_and_of_infinities():
    s = rotary_state(F32, 4, 2, 1, 64, 64, True, False)
    s["q"][1] = 0
    s["q"][2, 0, 5] = math.inf
    qo, ko = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    kw = dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=s["eps"])
    g.gpt2_op_qk_norm_rotary_forward(qo, ko, s["q"], s["k"], s["pos"], s["turns"], **kw)
    assert not qo[1].any() and torch.isfinite(qo[3]).all() and torch.isfinite(ko).all()
    assert torch.isfinite(qo[2, 1]).all()  # the other head of that row
    dq, dk, ones = torch.empty_like(qo), torch.empty_like(ko), torch.ones_like(qo)
    g.gpt2_op_qk_norm_rotary_backward(dq, dk, ones, torch.ones_like(ko), s["q"], s["k"], s["pos"], s["turns"], **kw)
    dx, _, bound, _ = R.rotary_backward(ones.double()[1:2], s["q"].double()[1:2], s["pos"][1:2], s["turns"],
                                        s["q_gamma"].double(), s["eps"])
    near(dq[1:2], dx, bound, "row of zeros")


def test_rotary_without_rows():
    s = rotary_state(BF, 0, 2, 1, 64, 64, True, False)
    dqg, dkg = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    kw = dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=s["eps"])
    g.gpt2_op_qk_norm_rotary_forward(s["q"], s["k"], s["q"], s["k"], s["pos"], s["turns"], **kw)
    g.gpt2_op_qk_norm_rotary_backward(s["q"], s["k"], s["q"], s["k"], s["q"], s["k"], s["pos"], s["turns"], dq_gamma=dqg,
                                      dk_gamma=dkg, **kw)
    assert not dqg.any() and not dkg.any()


def test_rotary_repeats_and_follows_graphs_and_streams():
    s = rotary_state(BF, 3000, 12, 12, 64, 64, True, True)
    out = [torch.empty(3000, 12, 64, dtype=BF, device="cuda") for _ in range(4)] + [torch.empty(64, device="cuda")
                                                                                   for _ in range(2)]
    dqo, dko = rnd(3000, 12, 64, dtype=BF), rnd(3000, 12, 64, dtype=BF)
    kw = dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=s["eps"])

    def run(stream=None):
        g.gpt2_op_qk_norm_rotary_forward(out[0], out[1], s["q"], s["k"], s["pos"], s["turns"], stream=stream, **kw)
        g.gpt2_op_qk_norm_rotary_backward(out[2], out[3], dqo, dko, s["q"], s["k"], s["pos"], s["turns"], dq_gamma=out[4],
                                          dk_gamma=out[5], stream=stream, **kw)
    run()
    first = [x.clone() for x in out]
    graph = captured(run)
    for x in out:
        x.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, first))
    for x in out:
        x.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, first))
    # the graph reads the positions of its replay
    s["pos"].add_(1)
    run()
    later = [x.clone() for x in out]
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, later)) and not torch.equal(out[0], first[0])


def test_rotary_of_rows_more_than_31_bits_apart():
    stride = (1 << 30) + 8
    buf = torch.zeros(2 * stride + 256, device="cuda", dtype=BF)
    q, k = buf.as_strided((3, 2, 64), (stride, 64, 1)), buf[128:].as_strided((3, 1, 64), (stride, 64, 1))
    a, b = rnd(3, 2, 64, dtype=BF), rnd(3, 1, 64, dtype=BF)
    q.copy_(a)
    k.copy_(b)
    pos, turns = torch.tensor([3, 70, 900], device="cuda").int(), g.gpt2_rotary_turns(64).cuda()
    g.gpt2_op_qk_norm_rotary_forward(q, k, q, k, pos, turns, eps=1e-5)
    for x, y in ((a, q), (b, k)):
        near(y, *R.rotary(x.double(), pos, turns, None, 1e-5), "far rows")
    da, db = rnd(3, 2, 64, dtype=BF), rnd(3, 1, 64, dtype=BF)
    q.copy_(da)
    k.copy_(db)
    g.gpt2_op_qk_norm_rotary_backward(q, k, q, k, a, b, pos, turns, eps=1e-5)
    for dy, x, y in ((da, a, q), (db, b, k)):
        dx, _, bound, _ = R.rotary_backward(dy.double(), x.double(), pos, turns, None, 1e-5)
        near(y, dx, bound, "far rows")


# ---------------------------------------------------------------- cross entropy of hidden states

def hidden(N, C, V, Vp=None, dtype=BF, std=2.5):
    Vp = Vp or (V + 7) // 8 * 8
    w = torch.empty(Vp, C, device="cuda", dtype=dtype)
    w.copy_(rnd(Vp, C, std=std / math.sqrt(C)))
    w[V:] = math.nan  # what is padded is not used
    return rnd(N, C, dtype=dtype), w, torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)


def forward(x, w, t, V, **kw):
    losses, lse = torch.full((len(x),), math.nan, device="cuda"), torch.full((len(x),), math.nan, device="cuda")
    g.gpt2_op_linear_classifier_forward(losses, lse, x, w, t, V, **kw)
    return losses, lse


def classifier_case(N, C, V, dtype, dw_dtype=None, Vp=None, dlse=True, std=2.5):
    x, w, t = hidden(N, C, V, Vp, dtype, std)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses, lse = forward(x, w, t, V, status=status)
    want = R.classifier(x.double(), w.double(), t, V)
    near(losses, want[0], want[2], "losses")
    near(lse, want[1], want[3], "lse")
    assert (losses >= 0).all()
    d = torch.where(torch.rand(N, device="cuda") < 0.3, 0.0, rnd(N) / N)
    e = torch.where(d == 0, 0.0, 0.1 * rnd(N) / N) if dlse else None
    dx = torch.full_like(x, math.nan)
    dw = torch.full((w.shape[0], C), math.nan, device="cuda", dtype=dw_dtype or dtype)
    g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, V, dloss=d, dlse=e, status=status)
    rx, rw, bx, bw = R.classifier_backward(x.double(), w.double(), t, V, d.double(), e.double() if dlse else None, dtype)
    near(dx, rx, bx, "dx")
    near(dw[:V], rw, bw, "dw")
    assert not dw[V:].any() and status.item() == 0
    assert not dx[d == 0].any()


@pytest.mark.parametrize("dtype,dw_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("N,C,V", [(1, 8, 1), (1, 64, 50), (7, 72, 129), (128, 64, 256), (129, 200, 1000), (61, 768, 5003),
                                   (513, 128, 777), (700, 64, 2049), (1030, 1600, 1100)])
def test_classifier(dtype, dw_dtype, N, C, V):
    classifier_case(N, C, V, dtype, dw_dtype)


@pytest.fixture
def pieces_of_256_mb():
    lib = g.load_library()
    g.check(lib.gpt2_debug_linear_classifier_piece(256 << 20))
    yield
    g.check(lib.gpt2_debug_linear_classifier_piece(0))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_classifier_in_pieces(dtype, pieces_of_256_mb):
    # 70000 rows: pieces of 2048 columns, the last of them ragged
    classifier_case(70000, 16, 4357, dtype, F32, Vp=4400)


@pytest.mark.parametrize("C", [768, 1024, 640])
def test_classifier_adds_dx_from_piece_to_piece(C, pieces_of_256_mb):
    # two pieces; dx in 192-wide tiles of CTA pairs, in 256-wide ones, in tiles of one CTA
    classifier_case(8192, C, 17001, BF, BF, dlse=False)


@pytest.mark.parametrize("C", [768, 1024])
def test_classifier_of_many_rows_at_once(C):
    # one piece: dx and dw straight from 192-wide and 256-wide tiles of CTA pairs
    classifier_case(8192, C, 9001, BF, BF, Vp=9216, dlse=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [300, 2048, 2049, 40000, 70001])
def test_classifier_of_means_over_any_number(N, dtype):
    # 1 / N in every row, which bf16 does not hold: the gradients are off by their values' own roundings only
    C, V = 64, 100
    x, w, t = hidden(N, C, V, 104, dtype)
    _, lse = forward(x, w, t, V)
    d = torch.full((N,), 1.0 / N, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(104, C, device="cuda")
    g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, V, dloss=d)
    rx, rw, _, _ = R.classifier_backward(x.double(), w.double(), t, V, d.double(), None, dtype)
    # the sum of dw over the vocabulary's rows along the gradient itself: a common factor would show
    along = ((dw[:V].double() * rw).sum() / (rw * rw).sum()).item()
    # roundings of 100 N values of dz, none off by more than 2^-8 and of either sign: 2^-8 / sqrt(3) / sqrt(N) at most
    # of each row's largest, five times that, and fp32 sums
    assert abs(along - 1) < 5 * (2.0 ** -8 if dtype is BF else 2.0 ** -20) / math.sqrt(3 * N) + 2e-6


def test_classifier_of_the_models_vocabulary():
    classifier_case(300, 768, 50257, BF, BF, Vp=50304)


def test_classifier_accumulates():
    N, C, V = 200, 64, 1003
    x, w, t = hidden(N, C, V, 1008)
    _, lse = forward(x, w, t, V)
    d = rnd(N)
    dx, once, start = torch.empty_like(x), torch.empty(1008, C, device="cuda"), rnd(1008, C)
    g.gpt2_op_linear_classifier_backward(dx, once, x, w, t, lse, V, dloss=d)
    twice = start.clone()
    g.gpt2_op_linear_classifier_backward(dx, twice, x, w, t, lse, V, dloss=d, accumulate=True)
    near(twice[:V], start[:V].double() + once[:V].double(), once[:V].double().abs() * 4 * R.U * 16 + start[:V].abs() * R.U * 4,
         "dw added to")
    assert torch.equal(twice[V:], start[V:])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_classifier_of_sure_tokens_far_from_zero(dtype):
    # logits near 1000 for every token, the target 200 above them: the loss is 0, not the rounding of 1200
    N, C, V = 40, 64, 300
    x = torch.zeros(N, C, device="cuda", dtype=dtype)
    x[:, 0], x[:, 1] = 32.0, 1.0
    w = torch.zeros(304, C, device="cuda", dtype=dtype)
    w[:, 0] = 31.25
    w[:V, 1] = torch.linspace(-4, 4, V, device="cuda")
    t = torch.arange(N, device="cuda", dtype=torch.int32) * 7
    x[torch.arange(N), 2 + torch.arange(N, device="cuda") % 60] = 16.0
    w[t.long(), 2 + torch.arange(N, device="cuda") % 60] = 12.5
    losses, lse = forward(x, w, t, V)
    want = R.classifier(x.double(), w.double(), t, V)
    # these logits are exact in fp32 where the sums of their products are: all that is left is the final arithmetic
    assert (losses >= 0).all() and (losses.double() - want[0]).abs().max() < 1e-6
    assert ((lse.double() - want[1]).abs() <= 2 * R.U * want[1].abs()).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_classifier_targets_out_of_range(dtype):
    N, C, V = 130, 64, 100
    x, w, t = hidden(N, C, V, 104, dtype)
    t[3], t[129] = -1, V
    ok = t.clone()
    ok[3] = ok[129] = 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses, lse = forward(x, w, t, V, status=status)
    assert status.item() == 4
    again = forward(x, w, ok, V)
    assert torch.equal(losses, again[0]) and torch.equal(lse, again[1])
    status.zero_()
    out = []
    for tt, st in ((t, status), (ok, None)):
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        g.gpt2_op_linear_classifier_backward(dx, dw, x, w, tt, lse, V, dloss=torch.ones(N, device="cuda"), status=st)
        out.append((dx, dw))
    assert status.item() == 4 and torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_classifier_rows_that_do_not_count(dtype):
    N, C, V = 300, 64, 500
    x, w, t = hidden(N, C, V, 504, dtype)
    _, lse = forward(x, w, t, V)
    d = rnd(N)
    d[100:200] = 0
    lse[100:150] = math.nan  # of padding: never computed
    lse[150:200] = -math.inf
    dx, dw = torch.empty_like(x), torch.empty(504, C, device="cuda")
    g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, V, dloss=d)
    assert not dx[100:200].any() and torch.isfinite(dw).all()
    x2 = torch.cat((x[:100], x[200:]))
    rx, rw, bx, bw = R.classifier_backward(x2.double(), w.double(), torch.cat((t[:100], t[200:])), V,
                                           torch.cat((d[:100], d[200:])).double(), None, dtype)
    near(torch.cat((dx[:100], dx[200:])), rx, bx, "dx")
    near(dw[:V], rw, bw * 2, "dw")  # (n of the bound: the rows with zeros are added too)


def test_classifier_without_gradients_and_rows():
    x, w, t = hidden(5, 64, 50, 56)
    _, lse = forward(x, w, t, 50)
    dx, dw = torch.ones_like(x), torch.ones_like(w)
    g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, 50)
    assert not dx.any() and not dw.any()
    x, t, none = x[:0], t[:0], torch.empty(0, device="cuda")
    g.gpt2_op_linear_classifier_forward(none, none, x, w, t, 50)
    dw.fill_(1)
    g.gpt2_op_linear_classifier_backward(x, dw, x, w, t, none, 50)
    assert not dw.any()
    keep = torch.ones(56, 64, device="cuda")
    g.gpt2_op_linear_classifier_backward(x, keep, x, w, t, none, 50, accumulate=True)
    assert (keep == 1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_classifier_agrees_with_the_separate_operators(dtype):
    # the head's matmul and the classifier on its logits, as the step runs them
    N, C, V, Vp = 256, 128, 1000, 1024
    x, w, t = hidden(N, C, V, Vp, dtype)
    w[V:] = 0
    z = torch.empty(N, Vp, device="cuda", dtype=dtype)
    g.gpt2_op_matmul(z, x, 0, w, 0, N, Vp, C)
    losses = torch.empty(N, device="cuda")
    g.gpt2_op_classifier(z, losses, t, V, 1.0 / N)
    got, lse = forward(x, w, t, V)
    # each logit of the separate operators is rounded to their type
    top = (x.double() @ w.double().T).abs().amax(1)
    assert ((got - losses).abs() <= 2.2 * R.HALF[dtype] * top + 1e-5).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_classifier_repeats_and_follows_graphs_and_streams(dtype):
    N, C, V = 700, 64, 3001
    x, w, t = hidden(N, C, V, 3008, dtype)
    losses, lse, d = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), rnd(N)
    dx, dw = torch.empty_like(x), torch.empty(3008, C, device="cuda")

    def run(stream=None):
        g.gpt2_op_linear_classifier_forward(losses, lse, x, w, t, V, stream=stream)
        g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, V, dloss=d, stream=stream)
    out = (losses, lse, dx, dw)
    run()
    first = [o.clone() for o in out]
    graph = captured(run)
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    for o in out:
        o.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_classifier_reports_a_wait_that_runs_out():
    x, w, t = hidden(200, 64, 500, 504)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib = g.load_library()
    right = forward(x, w, t, 500)
    try:
        g.check(lib.gpt2_debug_set_wait_limit(2_000_000))
        g.check(lib.gpt2_debug_stall_matmul(1))
        forward(x, w, t, 500, status=status)
        torch.cuda.synchronize()
    finally:
        g.check(lib.gpt2_debug_stall_matmul(0))
        g.check(lib.gpt2_debug_set_wait_limit(0))
    assert status.item() & 2
    again = forward(x, w, t, 500)
    assert torch.equal(right[0], again[0]) and torch.equal(right[1], again[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_classifier_with_logits_of_minus_infinity(dtype):
    N, C, V = 20, 64, 300
    x, w, t = hidden(N, C, V, 304, dtype)
    x = x.abs() + 1
    w[40:200] = -math.inf  # whole chunks of the vocabulary
    t.copy_(torch.arange(N))
    t[7] = 60
    losses, lse = forward(x, w, t, V)
    keep = torch.cat((w[:40], w[200:V]))
    want = R.classifier(x.double(), keep.double(), t, len(keep))
    ok = torch.arange(N, device="cuda") != 7
    near(losses[ok], want[0][ok], want[2][ok], "losses")
    near(lse, want[1], want[3], "lse")
    assert losses[7] == math.inf
    w[:V] = -math.inf
    losses, lse = forward(x, w, t, V)
    assert (losses == math.inf).all() and (lse == -math.inf).all()
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, V, dloss=torch.ones(N, device="cuda"))
    assert not dw.any()
    for bad in (math.nan, math.inf):
        x, w, t = hidden(N, C, V, 304, dtype)
        x[3, 5] = bad
        losses, lse = forward(x, w, t, V)
        assert torch.isnan(losses[3]) and torch.isnan(lse[3])
        assert torch.isfinite(losses[:3]).all() and torch.isfinite(losses[4:]).all()


def test_classifier_of_more_values_than_31_bits():
    # dz has 2^31 values and more, the statistics 4 GB; rows from both ends and the middle are looked at
    N, C, V = (1 << 27) + 5, 8, 15
    x = torch.randint(-8, 9, (N, C), device="cuda", dtype=torch.int8).to(BF)
    _, w, _ = hidden(1, C, V, 16)
    t = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    losses, lse = forward(x, w, t, V)
    d = torch.zeros(N, device="cuda")
    at = torch.tensor([0, 1, 127, 128, N // 2, (1 << 26) + 3, N - 130, N - 2, N - 1], device="cuda")
    d[at] = 1.0
    dx, dw = torch.full_like(x, math.nan), torch.empty(16, C, device="cuda")
    g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, V, dloss=d)
    want = R.classifier(x[at].double(), w.double(), t[at], V)
    near(losses[at], want[0], want[2], "losses")
    near(lse[at], want[1], want[3], "lse")
    rx, rw, bx, bw = R.classifier_backward(x[at].double(), w.double(), t[at], V, d[at].double(), None, BF)
    near(dx[at], rx, bx, "dx")
    near(dw[:V], rw, bw, "dw")  # (the other rows add zeros)
    dx[at] = 0
    assert not dx.any()


def test_classifier_graphs_that_share_a_pool():
    V, pool, graphs = 777, torch.cuda.graph_pool_handle(), []
    for N, C in ((300, 64), (700, 128)):
        x, w, t = hidden(N, C, V, 784)
        out = [torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), torch.empty_like(x), torch.empty_like(w)]
        d = rnd(N)

        def run(x=x, w=w, t=t, out=out, d=d):
            g.gpt2_op_linear_classifier_forward(out[0], out[1], x, w, t, V)
            g.gpt2_op_linear_classifier_backward(out[2], out[3], x, w, t, out[1], V, dloss=d)
        run()
        first = [o.clone() for o in out]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            run()
        graphs.append((graph, out, first, run))  # (run holds the operands that the graph reads)
    for _ in range(3):
        for graph, out, *_ in graphs:
            for o in out:
                o.zero_()
            graph.replay()
        for _, out, first, _ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, first))


# ---------------------------------------------------------------- AdamW over many tensors

HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)


def tensors(sizes, bits, grads=F32, offset=0, zero=False):
    """Tensors of these sizes, each starting `offset` values into its own buffer, guarded by what lies around it."""
    def one(n, make, dtype):
        buf = torch.full((n + offset + 32,), 77.0, device="cuda").to(dtype)
        buf[offset:offset + n] = make(n)
        return buf[offset:offset + n]
    s = {"masters": [one(n, lambda n: rnd(n, std=0.1), F32) for n in sizes],
         "grads": [one(n, lambda n: rnd(n, std=10.0 ** (i % 4 - 3)), grads) for i, n in enumerate(sizes)],
         "params": [one(n, lambda n: torch.zeros(n, device="cuda"), BF) for n in sizes],
         "weight_decay": [0.1 * (i % 3) for i in range(len(sizes))]}
    if bits == 32:
        s["ms"] = [one(n, lambda n: torch.zeros(n, device="cuda") if zero else rnd(n, std=1e-2), F32) for n in sizes]
        s["vs"] = [one(n, lambda n: torch.zeros(n, device="cuda") if zero else rnd(n, std=1e-2).square(), F32)
                   for n in sizes]
        return s
    u8 = torch.uint8
    code = lambda top: lambda n: (torch.zeros(n, device="cuda", dtype=u8) if zero else  # noqa: E731
                                  torch.randint(0, top, (n,), device="cuda").to(u8))
    scale = lambda lo: lambda n: (torch.zeros(n, device="cuda", dtype=u8) if zero else  # noqa: E731
                                  torch.randint(lo, lo + 6, (n,), device="cuda").to(u8))
    s["ms"] = [one(n, code(0x79), u8) for n in sizes]
    s["vs"] = [one(n, code(0xF1), u8) for n in sizes]
    blocks = [-(-n // 128) for n in sizes]
    s["m_scales"] = [one(n, scale(112), u8) for n in blocks]
    s["v_scales"] = [one(n, scale(100), u8) for n in blocks]
    s["m_values"], s["v_values"] = ([torch.full((n,), math.nan, device="cuda") for n in sizes] for _ in range(2))
    return s


def held(s):
    return {k: [x.clone() for x in v] for k, v in s.items() if k != "weight_decay"}


def compare(before, s, t, factor, seed=0, start=0):
    """Every tensor of s (from its start-th value on) after step t against the oracle's step from `before`."""
    eight = "m_scales" in s
    for i, master in enumerate(s["masters"]):
        n = master.numel()
        if eight:
            m0, v0 = (R.values(before[a][i], before[b][i], k) for a, b, k in (("ms", "m_scales", "m"),
                                                                             ("vs", "v_scales", "v")))
        else:
            m0, v0 = before["ms"][i].double(), before["vs"][i].double()
        th0, gr = before["masters"][i].double(), before["grads"][i].double() * factor
        th, m, v = R.adamw(th0, before["grads"][i].double(), m0, v0, wd=s["weight_decay"][i], t=t, factor=factor,
                           lr=HP["lr"], b1=HP["beta1"], b2=HP["beta2"], eps=HP["eps"])
        # a product each for grad_scale and clip, two products and a sum for a moment (the clip's own 8 U among them)
        em, ev = 14 * R.U * (m0.abs() + gr.abs()), 26 * R.U * v
        step = (th - th0).abs() + HP["lr"] * s["weight_decay"][i] * th0.abs()
        slope = HP["lr"] * em / (1 - HP["beta1"] ** t) / (torch.sqrt(v / (1 - HP["beta2"] ** t)) + HP["eps"])
        eth = slope + 40 * R.U * (step + HP["lr"] * (m / (1 - HP["beta1"] ** t)).abs()
                                  / (torch.sqrt(v / (1 - HP["beta2"] ** t)) + HP["eps"])) + 2 * R.U * th.abs()
        near(master, th, eth, f"master {i}")
        if s["params"][i] is not None:
            assert torch.equal(s["params"][i], master.to(BF))
        if not eight:
            near(s["ms"][i], m, em, f"m {i}")
            near(s["vs"][i], v, ev, f"v {i}")
            continue
        for x, ex, code, scale, kind, u in zip((m, v), (em, ev), ("ms", "vs"), ("m_scales", "v_scales"), "mv",
                                               R.draws(n, i, t, seed, "cuda", start)):
            sc = s[scale][i].long()
            lo, hi = R.scales(x.abs() - ex, kind), R.scales(x.abs() + ex, kind)
            assert ((lo <= sc) & (sc <= hi)).all(), f"scale of {kind} {i}"
            got = R.values(s[code][i], s[scale][i], kind)
            unit = torch.exp2(sc[torch.arange(n, device="cuda") // 128].double() - 127)
            # in codes: the value's own error at 16 codes a binade, and the draw's 2^-16
            slack = 2.0 ** -14 + (ex / unit * 2.0 ** (9 if kind == "m" else 17)).clamp_max(1.0)
            slack = torch.where(x.abs() / unit >= 2.0 ** (-6 if kind == "m" else -14), 2.0 ** -14 + 16 * ex / x.abs(), slack)
            a, b = (R.stored(x, sc, u, kind, off) for off in (-slack, slack))
            low, high = torch.minimum(a, b), torch.maximum(a, b)
            assert ((low <= got) & (got <= high)).all(), f"{kind} {i}"
            assert ((a == b).float().mean() > 0.98) or n < 200


SIZES = [[1], [127, 128, 129], [4096, 4097, 5, 0, 12288, 3], [100003], [0, 0], list(range(1, 60)),
         [(i * 37) % 300 for i in range(391)]]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grads", [F32, BF])
@pytest.mark.parametrize("k", range(len(SIZES)))
def test_adamw_many(bits, grads, k):
    offset = 0 if k % 2 else 1 + k  # aligned and not
    s = tensors(SIZES[k], bits, grads, offset)
    h = g.gpt2_adamw_tensors(**s)
    for t, clip in ((1, 0.0), (7, 0.5), (1000, 1e9)):
        before = held(s)
        norm = torch.full((1,), math.nan, device="cuda")
        g.gpt2_op_adamw_many(h, **HP, t=t, grad_scale=0.25, max_grad_norm=clip, grad_norm=norm, seed=99 + k)
        want = math.sqrt(sum(x.double().square().sum().item() for x in before["grads"]))
        assert abs(norm.item() - want) <= 600 * R.U * want  # sums of 16 squares a thread, then in a tree
        factor = 0.25 * (min(1.0, clip / (want * 0.25 + 1e-6)) if clip else 1.0)
        compare(before, s, t, factor, 99 + k)
        for name, xs in s.items():  # what lies around the tensors
            if name not in ("weight_decay", "m_values", "v_values"):
                for x in xs:
                    around = x._base
                    assert (around[:offset] == 77).all() and (around[offset + x.numel():] == 77).all(), name
    if bits == 8:
        g.gpt2_op_adamw_many_states(h)
        for i in range(len(SIZES[k])):
            for code, scale, value, kind in (("ms", "m_scales", "m_values", "m"), ("vs", "v_scales", "v_values", "v")):
                assert torch.equal(s[value][i].double(), R.values(s[code][i], s[scale][i], kind))


def test_adamw_many_is_the_single_operator_for_each_tensor():
    s = tensors([4096, 64, 100000], 32)
    one = held(s)
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**s), **HP, t=3)
    for i, wd in enumerate(s["weight_decay"]):
        a = {k: v[i].clone() for k, v in one.items()}
        g.gpt2_op_adamw(a["masters"], a["params"], a["grads"], a["ms"], a["vs"], HP["lr"], HP["beta1"], HP["beta2"],
                        HP["eps"], wd, 3)
        for k in ("masters", "params", "ms", "vs"):
            assert torch.equal(a[k], s[k][i]), k


def test_adamw_many_from_zero_moments_and_without_copies():
    for bits in (8, 32):
        s = tensors([1000, 130], bits, zero=True)
        s["params"][1] = None
        before = {k: [x.clone() if x is not None else None for x in v] for k, v in s.items() if k != "weight_decay"}
        g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**s), **HP, t=1, seed=5)
        compare(before, s, 1, 1.0, 5)


def test_adamw_many_without_gradients_keeps_zero_moments():
    s = tensors([500], 8, zero=True)
    s["grads"][0].zero_()
    s["weight_decay"] = [0.0]
    before = held(s)
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**s), **HP, t=1)
    assert torch.equal(s["masters"][0], before["masters"][0]) and not s["ms"][0].any() and not s["vs"][0].any()


def test_adamw_many_keeps_a_nan_to_itself():
    for bits in (8, 32):
        s = tensors([700], bits)
        s["grads"][0][5], s["grads"][0][300] = math.nan, math.inf
        before = held(s)
        g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**s), **HP, t=2, seed=1)
        bad = torch.zeros(700, dtype=torch.bool, device="cuda")
        bad[5] = bad[300] = True
        assert torch.isnan(s["masters"][0][bad]).all() and torch.isfinite(s["masters"][0][~bad]).all()
        if bits == 8:
            assert (s["ms"][0][bad] & 0x7F == 0x7F).all() and (s["vs"][0][bad] == 0xFF).all()
            v = R.values(s["vs"][0], s["v_scales"][0], "v")
            assert torch.isfinite(v[~bad]).all()
            clean = {k: [x.clone() for x in xs] for k, xs in before.items()}
            clean["grads"][0][bad] = 0
            clean |= {"weight_decay": s["weight_decay"]}
            g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**clean), **HP, t=2, seed=1)
            same = ~bad
            blocks = [b for b in range(6) if b not in (0, 2)]
            for b in blocks:  # the other blocks hold the same bits
                at = slice(b * 128, (b + 1) * 128)
                assert torch.equal(clean["ms"][0][at], s["ms"][0][at]) and torch.equal(clean["vs"][0][at], s["vs"][0][at])
            assert torch.equal(clean["masters"][0][same], s["masters"][0][same])


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_many_of_more_values_than_31_bits(bits):
    n, tail = (1 << 31) + 4096 + 77, 3 * 128 + 77
    moment, kw = (torch.uint8 if bits == 8 else F32), dict(device="cuda")
    s = {"masters": [torch.zeros(n, **kw)], "grads": [torch.zeros(n, dtype=BF, **kw)], "weight_decay": [0.1],
         "ms": [torch.zeros(n, dtype=moment, **kw)], "vs": [torch.zeros(n, dtype=moment, **kw)], "params": [None]}
    if bits == 8:
        s |= {k: [torch.zeros(-(-n // 128), dtype=torch.uint8, **kw)] for k in ("m_scales", "v_scales")}
    s["masters"][0][-tail:] = rnd(tail)
    s["grads"][0][-tail:] = rnd(tail)
    h = g.gpt2_adamw_tensors(**s)
    ends = lambda s: {k: [x if x is None else x[-(4 if k.endswith("scales") else tail):].clone() for x in v]  # noqa: E731
                      if k != "weight_decay" else v for k, v in s.items()}
    before = ends(s)
    norm = torch.empty(1, **kw)
    g.gpt2_op_adamw_many(h, **HP, t=3, max_grad_norm=2.0, grad_norm=norm, seed=4)
    want = before["grads"][0].double().norm().item()
    assert abs(norm.item() - want) <= 600 * R.U * want
    compare(before, ends(s), 3, 2.0 / (want + 1e-6), 4, start=n - tail)
    assert not s["masters"][0][:-tail].any() and not s["ms"][0][:-tail].any()


@pytest.mark.parametrize("grads", [F32, BF])
def test_eight_bit_codes_are_those_of_plain_fp32_steps(grads):
    # each product and sum rounded on its own, the norm to its last bit: elementary fp32 operations give the same codes
    s = tensors([200001, 3000], 8, grads)
    h = g.gpt2_adamw_tensors(**s)
    f = lambda x: torch.tensor(x, dtype=F32, device="cuda")  # noqa: E731
    for t in (1, 2, 3):
        before = held(s)
        g.gpt2_op_adamw_many(h, **HP, t=t, grad_scale=0.25, max_grad_norm=0.5, seed=21)
        norm = sum(x.double().square().sum() for x in before["grads"]).sqrt().float()
        scale = f(0.25) * (f(0.5) / (norm * f(0.25) + f(1e-6))).clamp_max(1.0)
        for i in range(2):
            gr = before["grads"][i].float() * scale
            b1, b2 = f(HP["beta1"]), f(HP["beta2"])
            m0, v0 = (R.values(before[a][i], before[b][i], k).float() for a, b, k in (("ms", "m_scales", "m"),
                                                                                     ("vs", "v_scales", "v")))
            m, v = b1 * m0 + (1 - b1) * gr, b2 * v0 + (1 - b2) * (gr * gr)
            for x, u, code, sc, kind in zip((m, v), R.draws(gr.numel(), i, t, 21, "cuda"), ("ms", "vs"),
                                            ("m_scales", "v_scales"), "mv"):
                assert torch.equal(s[sc][i].long(), R.scales(x.double(), kind))
                got, want = R.values(s[code][i], s[sc][i], kind), R.stored(x.double(), s[sc][i].long(), u, kind)
                unit = torch.exp2(s[sc][i].double() - 127)[torch.arange(len(x), device="cuda") // 128]
                lowest = unit * 2.0 ** (-6 if kind == "m" else -14)  # (below it the code's own arithmetic rounds)
                assert ((got == want) | (x.double().abs() < lowest)).all() and (got != want).sum() < 5


def test_eight_bit_moments_follow_the_gradients_size():
    # gradients of one size for long, then of a tenth of it: v comes down too, which nearest rounding would not let it
    n = 4096
    s = tensors([n], 8, zero=True)
    h = g.gpt2_adamw_tensors(**s)
    hp = dict(lr=0.0, beta1=0.9, beta2=0.99, eps=1e-8)
    for t in range(1, 1401):
        s["grads"][0].copy_(rnd(n) * (1.0 if t <= 600 else 0.1))
        g.gpt2_op_adamw_many(h, **hp, t=t, seed=3)
        if t == 600:
            g.gpt2_op_adamw_many_states(h)
            high = s["v_values"][0].double().mean().item()
    g.gpt2_op_adamw_many_states(h)
    low = s["v_values"][0].double().mean().item()
    # the means of 4096 values: each v has a relative spread of sqrt(2 (1 - b2) / (1 + b2)) = 0.1 from its gradients, and
    # less than 0.3 from the rounding (steps of at most 1/8 once in about ten, over 100): 0.32 / 64 = 0.005; five of them
    assert abs(high - 1.0) < 0.025 and abs(low / 0.01 - 1.0) < 0.06  # (what is left of the first size: 0.99^800 * 100 = 0.032)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_many_repeats_and_follows_graphs_and_streams(bits):
    s = tensors([5000, 77, 40000], bits)
    start = held(s)
    h = g.gpt2_adamw_tensors(**s)
    norm = torch.empty(1, device="cuda")
    written = [x for k in ("masters", "params", "ms", "vs", "m_scales", "v_scales") for x in s.get(k, [])]

    def restore():
        for k, xs in start.items():
            for a, b in zip(s[k], xs):
                a.copy_(b)

    def run(stream=None):
        g.gpt2_op_adamw_many(h, **HP, t=4, max_grad_norm=0.3, grad_norm=norm, seed=8, stream=stream)
    run()
    first = [x.clone() for x in written]
    graph = captured(run)
    restore()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(written, first))
    restore()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(written, first))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grads", [F32, BF])
@pytest.mark.parametrize("far", [math.inf, -math.inf, 1e30])
def test_adamw_many_clips_by_an_infinite_norm(far, grads, bits):
    """Gradients whose squares' sum is no fp32 number clip all finite ones to 0."""
    s = tensors([20000, 700], bits, grads)
    s["grads"][0][9000] = far
    clean = held(s) | {"weight_decay": s["weight_decay"]}
    norm = torch.zeros(1, device="cuda")
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**s), **HP, t=2, seed=1, max_grad_norm=1.0, grad_norm=norm)
    assert norm.item() == math.inf
    for x in clean["grads"]:
        x.zero_()
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**clean), **HP, t=2, seed=1)
    for k in ("masters", "params", "ms", "vs"):
        for i, (a, b) in enumerate(zip(s[k], clean[k])):
            same = torch.ones(a.numel(), dtype=torch.bool, device="cuda")
            if math.isinf(far) and i == 0:  # inf * 0 is NaN, where it is; the block's scale is that of the other values
                same[9000 // 128 * 128:(9000 // 128 + 1) * 128] = bits == 32 or k in ("masters", "params")
                same[9000] = False
            assert torch.equal(a[same], b[same]), (k, i)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_many_clips_a_negative_scale(bits):
    """grad_scale < 0 turns the gradients round, clipped or not."""
    s = tensors([5000, 700], bits)
    turned = held(s) | {"weight_decay": s["weight_decay"]}
    for x in turned["grads"]:
        x.neg_()
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**s), **HP, t=2, seed=1, max_grad_norm=0.5, grad_scale=-0.25)
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**turned), **HP, t=2, seed=1, max_grad_norm=0.5, grad_scale=0.25)
    for k in ("masters", "params", "ms", "vs"):
        assert all(torch.equal(a, b) for a, b in zip(s[k], turned[k])), k


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_on_two_streams_at_once(dtype):
    """Two programs of the same calls, several deep on a stream each, write what they write alone."""
    def program(rows, C, V):
        x, w, t = hidden(rows, C, V, dtype=dtype)
        s = rotary_state(dtype, rows, 4, 2, 64, 64, True, False)
        a = tensors([5000, 77, 40000], 8 if dtype is BF else 32)
        start, h = held(a), g.gpt2_adamw_tensors(**a)
        d, kw = rnd(rows), dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=s["eps"])
        out = [torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x), torch.empty_like(w),
               torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty(64, device="cuda"),
               torch.empty(64, device="cuda")]
        written = out + [y for k in ("masters", "params", "ms", "vs", "m_scales", "v_scales") for y in a.get(k, [])]

        def run():
            for k, ys in start.items():
                for y, was in zip(a[k], ys):
                    y.copy_(was)
            g.gpt2_op_linear_classifier_forward(out[0], out[1], x, w, t, V)
            g.gpt2_op_linear_classifier_backward(out[2], out[3], x, w, t, out[1], V, dloss=d)
            g.gpt2_op_qk_norm_rotary_backward(out[4], out[5], s["q"], s["k"], s["q"], s["k"], s["pos"], s["turns"],
                                              dq_gamma=out[6], dk_gamma=out[7], **kw)
            g.gpt2_op_adamw_many(h, **HP, t=4, max_grad_norm=0.3, seed=8)
        return run, written
    programs = [program(300, 64, 3001), program(700, 128, 1777)]
    alone = []
    for run, written in programs:
        run()
        alone.append([y.clone() for y in written])
    for _, written in programs:
        for y in written:
            y.zero_()
    streams = [torch.cuda.Stream() for _ in programs]
    torch.cuda.synchronize()
    for _ in range(8):
        for (run, _), stream in zip(programs, streams):
            with torch.cuda.stream(stream):
                run()
    torch.cuda.synchronize()
    for (_, written), want in zip(programs, alone):
        assert all(torch.equal(y, z) for y, z in zip(written, want))


def test_a_step_on_packed_documents():
    """Positions, attention over documents, the loss and the update, as a program runs them: the gradients against
    autograd in 64 bits, the update against the oracle."""
    lens, H, hd, V, Vp = [5, 130, 1, 64, 77], 4, 64, 300, 304
    C, n = H * hd, 280  # the last three rows are padding, of no document
    real = sum(lens)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    pos = torch.cat([torch.arange(x) for x in lens + [n - real]]).int().cuda()
    turns = g.gpt2_rotary_turns(hd).cuda()
    x = rnd(n, C, dtype=BF)
    wq, wh = rnd(3 * C, C, dtype=BF, std=0.06), rnd(Vp, C, dtype=BF, std=0.1)
    gq, gk = (1 + 0.1 * rnd(hd)).to(BF), (1 + 0.1 * rnd(hd)).to(BF)
    t = torch.randint(0, V, (n,), device="cuda").int()
    d = torch.full((n,), 1.0 / real, device="cuda")
    d[real:] = 0
    heads = lambda b, i: b[:, i * C:(i + 1) * C].unflatten(1, (H, hd))  # noqa: E731
    e = lambda *a, dtype=BF: torch.zeros(*a, device="cuda", dtype=dtype)  # noqa: E731

    qkv = e(n, 3 * C)
    g.gpt2_op_matmul(qkv, x, 0, wq, 0, n, 3 * C, C)
    q, k = e(n, H, hd), e(n, H, hd)
    kw = dict(q_gamma=gq, k_gamma=gk, eps=1e-6)
    g.gpt2_op_qk_norm_rotary_forward(q, k, heads(qkv, 0), heads(qkv, 1), pos, turns, **kw)
    o, alse = e(n, H, hd), e(H, n, dtype=F32)
    g.gpt2_op_attention_packed_forward(o, alse, q, k, heads(qkv, 2), cu, cu, max(lens), max(lens))
    hid, losses, lse = o.view(n, C), e(n, dtype=F32), e(n, dtype=F32)
    g.gpt2_op_linear_classifier_forward(losses, lse, hid, wh, t, V)
    do, dwh = e(n, C), e(Vp, C, dtype=F32)
    g.gpt2_op_linear_classifier_backward(do, dwh, hid, wh, t, lse, V, dloss=d)
    dqkv, dq, dk = e(n, 3 * C), e(n, H, hd), e(n, H, hd)
    g.gpt2_op_attention_packed_backward(dq, dk, heads(dqkv, 2), do.view(n, H, hd), q, k, heads(qkv, 2), o, alse, cu, cu,
                                        max(lens), max(lens))
    dgq, dgk = e(hd, dtype=F32), e(hd, dtype=F32)
    g.gpt2_op_qk_norm_rotary_backward(heads(dqkv, 0), heads(dqkv, 1), dq, dk, heads(qkv, 0), heads(qkv, 1), pos, turns,
                                      dq_gamma=dgq, dk_gamma=dgk, **kw)
    dwq = e(3 * C, C, dtype=F32)
    g.gpt2_op_matmul(dwq, dqkv, 1, x, 1, 3 * C, C, n)

    # in 64 bits
    leaves = [a.double().requires_grad_() for a in (wq, wh, gq, gk)]
    WQ, WH, GQ, GK = leaves
    QKV = x.double() @ WQ.T
    Q, K = (R.rotary(heads(QKV, i), pos, turns, gm, 1e-6)[0] for i, gm in ((0, GQ), (1, GK)))
    O = []
    for a, b in zip(cu.tolist(), cu.tolist()[1:]):
        s = torch.einsum("ihd,jhd->hij", Q[a:b], K[a:b]) / math.sqrt(hd)
        s = s.masked_fill(torch.ones(b - a, b - a, device="cuda", dtype=torch.bool).triu(1), -math.inf)
        O.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), heads(QKV, 2)[a:b]))
    loss = torch.nn.functional.cross_entropy(torch.cat(O).flatten(1) @ WH[:V].T, t.long()[:real])
    loss.backward()
    # seven roundings to bf16 on the way (qkv, q, k, o, dz, do, dq): half a step of 2^-8 each, and their sums' spread
    assert abs(losses[:real].double().mean() - loss) < 4 * 2.0 ** -8
    for got, leaf, name in ((dwh[:V], WH.grad[:V], "head"), (dwq, WQ.grad, "qkv"), (dgq, GQ.grad, "q_gamma"),
                            (dgk, GK.grad, "k_gamma")):
        rel = ((got.double() - leaf).norm() / leaf.norm()).item()
        assert rel < 7 * 2.0 ** -8, (name, rel)

    # the update of all of them, moments in 8 bits
    params = [wq, wh, gq, gk]
    s = {"masters": [p.float() for p in params], "grads": [dwq, dwh, dgq, dgk], "params": params,
         "ms": [torch.zeros_like(p, dtype=torch.uint8) for p in params],
         "vs": [torch.zeros_like(p, dtype=torch.uint8) for p in params], "weight_decay": [0.1, 0.1, 0.0, 0.0]}
    s |= {k: [torch.zeros(-(-p.numel() // 128), device="cuda", dtype=torch.uint8) for p in params]
          for k in ("m_scales", "v_scales")}
    before = held(s)
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**s), **HP, t=1, seed=2)
    flat = lambda s: {k: [x.reshape(-1) if torch.is_tensor(x) else x for x in v] for k, v in s.items()}  # noqa: E731
    compare(flat(before), flat(s), 1, 1.0, 2)
    # and the step went down the loss's slope
    assert sum(((b.double() - a.double()) * gr.double()).sum() for a, b, gr in zip(before["masters"], s["masters"],
                                                                                s["grads"])) < 0
