"""Calls at the edges of what packed attention and the token log-probabilities allow, against the float64 oracle."""
import numpy as np
import pytest

from oracle import packed_ref as P
from step_gpt_train_gb300 import data
from tests._gpu_util import dev, host, inputs
from tests.test_gpu_packed import Packed, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    from step_gpt_train_gb300 import gpt2 as g
    g.load_library(build=True)
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lq,hidden", [(300, 128), (200, 130), (200, 256), (1, 200)])
def test_attention_first_keys_score_minus_infinity(torch_cuda, lq, hidden, mode):
    """A query whose first keys all score -inf (products past fp32's range) is the query without them."""
    torch = torch_cuda
    lk = hidden + max(lq, 90)
    c = Packed(torch, 41, [lq], [lk], 4, 2, 64, mode, before=0, after=0)
    first = slice(0, hidden)
    c.q[..., 0] = float(data.round_to_bf16(np.float32([1e20]))[0])
    c.k[..., 0] = 0.0
    c.k[first, :, 0] = -c.q[0, 0, 0]
    c.tq.copy_(dev(c.q.astype(np.float32), mode))
    c.tk.copy_(dev(c.k.astype(np.float32), mode))
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    rest = slice(hidden, lk)
    cu_k = np.array([0, lk - hidden])
    o, lse, bo, bl = P.attention_forward(c.q, c.k[rest], c.v[rest], c.cu_q, cu_k, mode)
    within(host(c.o), o, bo, "o")
    within(host(c.lse), lse, bl, "lse")
    dq, dk, dv, bq, bk, bv = P.attention_backward(c.dout, c.q, c.k[rest], c.v[rest], c.cu_q, cu_k, mode)
    within(host(c.dq), dq, bq, "dq")
    within(host(c.dk)[rest], dk, bk, "dk")
    within(host(c.dv)[rest], dv, bv, "dv")
    assert not c.dk[first].any() and not c.dv[first].any()


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
def test_attention_runs_of_items_without_keys(torch_cuda, mode):
    """Many work items in a row that meet no key (longer than a processor's share of them), among some that do."""
    r = np.random.default_rng(5)
    lq = [int(x) for x in r.integers(1, 300, 900)]
    lk = [0] * len(lq)
    lk[100], lk[101], lk[500], lq[700], lk[700] = 200, 7, 40, 2000, 300
    c = Packed(torch_cuda, 47, lq, lk, 4, 2, 64, mode)
    c.forward()
    c.backward()
    c.check()


def test_attention_scores_that_grow_stay_below_the_wait_limit(torch_cuda):
    """Rows whose scores outgrow their first block's by far take no longer than a wait may: with the bound of every
    wait at about a millisecond a prompt of 4096 tokens of such rows is done, and right."""
    torch = torch_cuda
    from step_gpt_train_gb300.gpt2 import check, load_library
    c = Packed(torch, 42, [4096], [4096], 16, 4, 64, 1)
    c.q[c.real_q] = 0
    c.q[c.real_q, :, 0] = 8.0
    n = int(c.real_k.sum())
    c.k[c.real_k, :, 0] = data.round_to_bf16(np.linspace(-100, 100, n).astype(np.float32))[:, None]
    c.tq.copy_(dev(c.q.astype(np.float32)))
    c.tk.copy_(dev(c.k.astype(np.float32)))
    lib = load_library()
    try:
        check(lib.gpt2_debug_set_wait_limit(2_000_000), "gpt2_debug_set_wait_limit")
        c.forward()
        torch.cuda.synchronize()
    finally:
        check(lib.gpt2_debug_set_wait_limit(0), "gpt2_debug_set_wait_limit")
    c.check(back=False)


@pytest.mark.parametrize("mode,hd", [(0, 64), (0, 16), (1, 64)])
@pytest.mark.parametrize("group", [1, 4])
def test_attention_offsets_in_any_order_touch_nothing_outside(torch_cuda, group, mode, hd):
    """Offsets out of order or range set bit 8, and nothing around the outputs is written, whatever they are."""
    torch = torch_cuda
    r = np.random.default_rng(group)
    arrays = [[398, 102, 43, 244, 9, 194], [393, 0, 0, 0, 0, 393], [0, 300, 20, 380, 10, 393], [393, 300, 200, 100, 50, 0]]
    arrays += [r.integers(-5, 400, 6).tolist() for _ in range(12)]
    around = 4096
    c = Packed(torch, 49, [80, 80, 80, 80, 73], [80, 80, 80, 80, 73], group, 1, hd, mode, before=0, after=0)
    c.max_q = c.max_k = 400
    fine = lambda x: x[0] >= 0 and x[-1] <= 393 and x == sorted(x)  # noqa: E731
    held = {}

    def within_walls(t):  # a copy with `around` values of 7 on either side
        wall = torch.full((t.numel() + 2 * around,), 7.0, dtype=t.dtype, device="cuda")
        return wall, wall[around:-around].view(t.shape)
    for name in ("o", "lse", "dq", "dk", "dv"):
        held[name], x = within_walls(getattr(c, name))
        setattr(c, name, x)
    for cu in arrays:
        for q, k in ((cu, [0, 80, 160, 240, 320, 393]), ([0, 80, 160, 240, 320, 393], cu), (cu, cu)):
            c.dev_cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (q, k)]
            for run in (c.forward, c.backward):
                c.status.zero_()
                run()
                torch.cuda.synchronize()
                assert c.status.item() == (0 if fine(q) and fine(k) else 8), (q, k)
    for name, wall in held.items():
        assert (wall[:around] == 7).all() and (wall[-around:] == 7).all(), name


@pytest.mark.parametrize("group", [1, 4])
def test_attention_new_tokens_with_offsets_in_any_order(torch_cuda, group):
    """The same for the kernels of few queries, cut over the keys and (max_k of 128) not."""
    torch = torch_cuda
    r = np.random.default_rng(10 + group)
    around = 4096
    c = Packed(torch, 50, [2] * 6, [80, 80, 80, 80, 73, 4000], group, 1, 64, 1, before=0, after=0)
    c.max_q = 4
    wall = torch.full((c.o.numel() + 2 * around,), 7.0, dtype=torch.bfloat16, device="cuda")
    wall_lse = torch.full((c.lse.numel() + 2 * around,), 7.0, device="cuda")
    c.o, c.lse = wall[around:-around].view(c.o.shape), wall_lse[around:-around].view(c.lse.shape)
    for c.max_k in (128, 4393):
        for _ in range(20):
            q, k = r.permutation(13)[:7].tolist(), r.integers(-5, 4400, 7).tolist()
            assert q != sorted(q)
            c.dev_cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (q, k)]
            c.status.zero_()
            c.forward()
            torch.cuda.synchronize()
            assert c.status.item() == 8, (q, k)
    for w in (wall, wall_lse):
        assert (w[:around] == 7).all() and (w[-around:] == 7).all()


@pytest.mark.parametrize("n,Hq,Hkv", [(3, 2, 2), (3, 10, 2), (60, 10, 2), (60, 12, 12)])
def test_attention_some_sequences_grow(torch_cuda, n, Hq, Hkv):
    """Every other sequence's scores rise or fall by 100 over its length, the rest stay as they are; the same bits twice."""
    torch = torch_cuda
    r = np.random.default_rng(n)
    lk = [int(x) for x in r.integers(1, 700, n)]
    lk[1] = 1500
    lq = [int(r.integers(0, x + 2)) if i % 3 else x for i, x in enumerate(lk)]
    c = Packed(torch, 48, lq, lk, Hq, Hkv, 64, 1)
    for i in range(1, n, 2):
        a, b = (slice(int(x[i]), int(x[i + 1])) for x in (c.cu_q, c.cu_k))
        c.q[a, :, 0] = 8.0 if i % 4 == 1 else -8.0
        c.k[b, :, 0] = data.round_to_bf16(np.linspace(-50, 50, lk[i]).astype(np.float32))[:, None]
    c.tq.copy_(dev(c.q.astype(np.float32)))
    c.tk.copy_(dev(c.k.astype(np.float32)))
    c.forward()
    o, lse = c.o.clone(), c.lse.clone()
    c.forward()
    c.backward()
    c.check()
    assert torch.equal(o.nan_to_num(), c.o.nan_to_num()) and torch.equal(lse, c.lse)


def test_attention_growing_scores_in_graphs(torch_cuda):
    """Graphs whose calls go through their items twice, replayed in turn with eager calls and on two streams at once."""
    torch = torch_cuda
    cs = []
    for seed, n in ((55, 900), (56, 2000)):
        c = Packed(torch, seed, [n, 50], [n, 700], 8, 2, 64, 1)
        c.tq[c.cu_q[0]:c.cu_q[-1], :, 0] = 8.0
        c.tk[c.cu_k[0]:c.cu_k[-1], :, 0] = torch.linspace(-90, 90, n + 700, device="cuda")[:, None].bfloat16()
        c.forward()
        cs.append((c, c.o.clone(), c.lse.clone(), torch.cuda.CUDAGraph(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for c, _, _, graph, _ in cs:
        with torch.cuda.graph(graph):
            c.forward()
    for _ in range(3):
        for c, *_ in cs:
            c.o.fill_(c.FILL)
            c.lse.fill_(c.FILL)
        torch.cuda.synchronize()
        for c, _, _, graph, stream in cs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for c, o, lse, _, _ in cs:
            assert c.status.item() == 0 and torch.equal(c.o, o) and torch.equal(c.lse, lse)
            c.forward()
            torch.cuda.synchronize()
            assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


def test_attention_backward_positions_times_heads_past_31_bits(torch_cuda):
    """64 heads on one over 2^25 keys: key positions counted in (query, head) rows pass 2^31. Every key is seen by the
    one query with the same weight, so every row of dV is the same, and dK is 0."""
    torch = torch_cuda
    from step_gpt_train_gb300.gpt2 import gpt2_op_attention_packed_backward
    lk, H = (1 << 25) + 256, 64
    z = lambda n, h: torch.zeros(n, h, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, o, dq, dout = z(1, H), z(1, H), z(1, H), z(1, H)
    dout.fill_(1.0)
    k, dk, dv = z(lk, 1), z(lk, 1), z(lk, 1)
    dk.fill_(7.0)
    dv.fill_(7.0)
    lse = torch.full((H, 1), float(np.log(lk)), device="cuda")
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (1, lk))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gpt2_op_attention_packed_backward(dq, dk, dv, dout, q, k, k, o, lse, cu_q, cu_k, 1, lk, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    # P rounds to bf16, the sum of 64 equal terms and dV's own rounding add half a step each; lse is off by 2^-24 |lse|
    want = H / lk
    lo, hi = dv.min().item(), dv.max().item()
    assert want * (1 - 2.5 * P.BF16) <= lo and hi <= want * (1 + 2.5 * P.BF16), (lo, hi, want)
    assert not dk.any() and not dq.any()


def test_attention_backward_wide_groups_report_bad_offsets_without_queries(torch_cuda):
    torch = torch_cuda
    c = Packed(torch, 43, [0, 0, 0], [30, 20, 10], 128, 1, 64, 1, before=0, after=0)
    c.dev_cu[1] = torch.tensor([0, 50, 30, 60], dtype=torch.int32, device="cuda")
    c.max_k = 60
    c.backward()
    torch.cuda.synchronize()
    assert c.status.item() == 8


def sure_rows(mode, N, V, Vp):
    """Rows in which one token holds nearly everything, at offsets from 0 to beyond 10^4, of either sign."""
    r = np.random.default_rng(N + V)
    z = inputs(44, (N, Vp), 1.0, 0).astype(np.float64)
    offsets = np.array([0.0, 10.0, -10.0, 100.0, -100.0, 1000.0, -1000.0, 4000.0, 9000.0, -30000.0])
    top = r.integers(0, V, N)
    z[np.arange(N), top] = 45.0 + r.random(N)
    z += (offsets[np.arange(N) % 10] * (1 + r.random(N)))[:, None]
    z = data.round_to_bf16(z.astype(np.float32)).astype(np.float64) if mode == 1 else z.astype(np.float32).astype(np.float64)
    return z, top


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,V,k", [(30, 500, 0), (30, 500, 5), (3, 50257, 5), (3, 50257, 0), (60, 50257, 40), (200, 50257, 0),
                                   (700, 5003, 20), (700, 5003, 0)])
def test_logprobs_of_sure_tokens(torch_cuda, N, V, k, mode):
    """Log-probabilities keep their accuracy however far the logits are from 0: none is positive, no entropy negative."""
    from tests.test_gpu_packed import run_logprobs
    z, top = sure_rows(mode, N, V, -(-V // 8) * 8)
    t = np.where(np.arange(N) % 3 == 2, (top + 1) % V, top)
    _, _, logp, lse, ent, tl, ids, status = run_logprobs(torch_cuda, z, t, V, k, mode)
    ref = P.token_logprobs(z, t, V, k)
    m = z[:, :V].max(axis=1, keepdims=True)
    others = np.exp(z[:, :V] - m).sum(axis=1) - 1  # the weight beside the largest's
    # z - m rounds once (bf16 logits: not at all) and logp once; ln S is off by its largest term's exponential (2^-22)
    # and four roundings near 1, and by the others' weight where it is lost beside 1
    bound = lambda x: 2 * P.F32 * np.abs(x) + 8 * P.F32 + np.abs(others)  # noqa: E731
    assert status.item() == 0
    within(host(logp), ref[1], bound(ref[1]), "logp")
    within(host(lse), ref[0], P.F32 * np.abs(ref[0]) + bound(0), "lse")
    # entropy = ln S - T / S, T of the others' weight times their distance (at most 64, or 130 in steps of bf16)
    within(host(ent), ref[2], bound(0) + 400 * np.abs(others), "entropy")
    assert (host(logp) <= 0).all() and (host(ent) >= 0).all() and (host(tl) <= 0).all()
    if k:
        assert (ids.cpu().numpy() == ref[3]).all()
        within(host(tl), ref[4], 2 * P.F32 * np.abs(ref[4]) + 8 * P.F32 + np.abs(others)[:, None], "top")


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,hi", [(2100, 40), (9000, 4)], ids=["offsets searched in memory", "unsorted"])
def test_attention_thousands_of_sequences(torch_cuda, n, hi, mode):
    """More sequences than the sort keeps in shared memory, and more work items than it takes."""
    r = np.random.default_rng(n)
    lk = [int(x) for x in r.integers(0, hi + 1, n)]
    lq = [int(r.integers(0, x + 2)) for x in lk]
    lk[n // 2] = lq[n // 2] = 700
    c = Packed(torch_cuda, 45, lq, lk, 2, 1, 64, mode)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("n", [1500, 3000])
def test_attention_new_tokens_of_thousands_of_sequences(torch_cuda, n):
    r = np.random.default_rng(n)
    lk = [int(x) for x in r.integers(0, 30, n)]
    lk[7], lk[n - 5], lk[n // 3] = 3000, 2000, 0
    c = Packed(torch_cuda, 46, [int(x) for x in r.integers(0, 2, n)], lk, 8, 2, 64, 1)
    c.forward()
    c.check(back=False)


@pytest.mark.parametrize("lq,lk", [(200, 300000), (100000, 100000)])
def test_attention_waits_that_run_out(torch_cuda, lq, lk):
    """With the bound of the waits at nothing the long waits of a long sequence run out: the kernels report it, stop
    and give back what they hold, so that the same call right after is as before."""
    torch = torch_cuda
    from step_gpt_train_gb300 import gpt2 as g
    new = lambda n, seed: dev(inputs(seed, (n, 1, 64), 1.0, 1))  # noqa: E731
    q, k, v, dout = new(lq, 51), new(lk, 52), new(lk, 53), new(lq, 54)
    o, lse = torch.zeros_like(q), torch.zeros(1, lq, device="cuda")
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (lq, lk))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def forward():
        g.gpt2_op_attention_packed_forward(o, lse, q, k, v, cu_q, cu_k, lq, lk, status=status)

    def backward():
        g.gpt2_op_attention_packed_backward(dq, dk, dv, dout, q, k, v, o, lse, cu_q, cu_k, lq, lk, status=status)
    forward()
    backward()
    first = [x.clone() for x in (o, lse, dq, dk, dv)]
    assert status.item() == 0
    lib = g.load_library()
    for run in (forward, backward):
        for x, y in zip((o, lse), first):  # (the backward's inputs)
            x.copy_(y)
        try:
            g.check(lib.gpt2_debug_set_wait_limit(1), "gpt2_debug_set_wait_limit")
            run()
            torch.cuda.synchronize()
        finally:
            g.check(lib.gpt2_debug_set_wait_limit(0), "gpt2_debug_set_wait_limit")
        assert status.item() == 2
        status.zero_()
    forward()
    backward()
    torch.cuda.synchronize()
    assert status.item() == 0
    for x, y in zip((o, lse, dq, dk, dv), first):
        assert torch.equal(x, y)
