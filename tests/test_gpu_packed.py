"""Packed-sequence attention and token log-probabilities on the GPU against the
float64 oracle, element by element within bounds that the oracle derives from
the roundings a kernel makes (oracle/packed_ref.py)."""
import numpy as np
import pytest

from oracle import packed_ref as P
from step_gpt_train_gb300 import data
from tests._gpu_util import dev, host, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    from step_gpt_train_gb300 import gpt2 as g
    g.load_library(build=True)
    torch.cuda.set_device(0)
    return torch


def within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    inf = np.isinf(ref)
    assert (got[inf] == ref[inf]).all(), what
    err = np.abs(got[~inf] - ref[~inf])
    bad = ~(err <= bound[~inf])
    if bad.any():
        i = np.argmax(np.where(bad, err / bound[~inf], 0))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; worst {err[i]:.3g}, allowed "
                             f"{bound[~inf][i]:.3g}")


class Packed:
    """Packed sequences on the device with `before` and `after` rows of no sequence around them, filled with NaN;
    outputs start as `FILL` everywhere."""
    FILL = 7.0

    def __init__(self, torch, seed, lq, lk, Hq, Hkv, hd, mode, fused=False, before=3, after=5, scale=1.0):
        self.torch, self.mode, self.dims = torch, mode, (Hq, Hkv, hd)
        off = lambda x, b: (np.concatenate([[0], np.cumsum(x)]) + b).astype(np.int32)  # noqa: E731
        self.cu_q, self.cu_k = off(lq, before), off(lk, before)
        self.rows_q, self.rows_k = int(self.cu_q[-1]) + after, int(self.cu_k[-1]) + after
        self.max_q, self.max_k = max(lq, default=0), max(lk, default=0)
        real_q = np.zeros(self.rows_q, bool)
        real_k = np.zeros(self.rows_k, bool)
        real_q[self.cu_q[0]:self.cu_q[-1]] = True
        real_k[self.cu_k[0]:self.cu_k[-1]] = True
        self.real_q, self.real_k = real_q, real_k

        def rows(seed, real, heads, s=1.0):
            x = inputs(seed, (len(real), heads, hd), s, mode).astype(np.float64)
            x[~real] = np.nan
            return x
        self.q, self.dout = rows(seed, real_q, Hq, scale), rows(seed + 3, real_q, Hq)
        self.k, self.v = rows(seed + 1, real_k, Hkv), rows(seed + 2, real_k, Hkv)
        self.dev_cu = [torch.from_numpy(c).cuda() for c in (self.cu_q, self.cu_k)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def blocks(*xs):  # column blocks of one buffer, or buffers of their own
            ts = [dev(x.astype(np.float32).reshape(len(x), x.shape[1] * x.shape[2]), mode) for x in xs]
            if not fused:
                return [t.unflatten(1, (-1, hd)) for t in ts]
            buf = torch.cat([torch.full((len(xs[0]), 16), float("nan"), dtype=ts[0].dtype, device="cuda")] + ts, 1)
            out, at = [], 16
            for t in ts:
                out.append(buf[:, at:at + t.shape[1]].unflatten(1, (-1, hd)))
                at += t.shape[1]
            return out
        if fused and self.rows_q == self.rows_k:
            self.tq, self.tk, self.tv = blocks(self.q, self.k, self.v)
        else:
            (self.tq,), (self.tk, self.tv) = blocks(self.q), blocks(self.k, self.v)
        (self.tdout,) = blocks(self.dout)
        like = lambda n, h: torch.full((n, h, hd), self.FILL, dtype=self.tq.dtype, device="cuda")  # noqa: E731
        self.o, self.lse = like(self.rows_q, Hq), torch.full((Hq, self.rows_q), self.FILL, device="cuda")
        self.dq, self.dk, self.dv = like(self.rows_q, Hq), like(self.rows_k, Hkv), like(self.rows_k, Hkv)

    def forward(self, **kw):
        from step_gpt_train_gb300.gpt2 import gpt2_op_attention_packed_forward as f
        return f(self.o, self.lse, self.tq, self.tk, self.tv, *self.dev_cu, self.max_q, self.max_k,
                 status=self.status, **kw)

    def backward(self, **kw):
        from step_gpt_train_gb300.gpt2 import gpt2_op_attention_packed_backward as f
        return f(self.dq, self.dk, self.dv, self.tdout, self.tq, self.tk, self.tv, self.o, self.lse, *self.dev_cu,
                 self.max_q, self.max_k, status=self.status, **kw)

    def check(self, back=True):
        self.torch.cuda.synchronize()
        assert self.status.item() == 0
        rq, rk = self.real_q, self.real_k
        o, lse, bo, bl = P.attention_forward(self.q, self.k, self.v, self.cu_q, self.cu_k, self.mode)
        go, gl = host(self.o), host(self.lse)
        within(go[rq], o[rq], bo[rq], "o")
        within(gl[:, rq], lse[:, rq], bl[:, rq], "lse")
        assert (go[~rq] == self.FILL).all() and (gl[:, ~rq] == self.FILL).all()
        if not back:
            return
        refs = P.attention_backward(self.dout, self.q, self.k, self.v, self.cu_q, self.cu_k, self.mode)
        for name, real, ref, bound in (("dq", rq, refs[0], refs[3]), ("dk", rk, refs[1], refs[4]),
                                       ("dv", rk, refs[2], refs[5])):
            got = host(getattr(self, name))
            within(got[real], ref[real], bound[real], name)
            assert (got[~real] == self.FILL).all(), name


CASES = {
    "one token": ([1], [1], 2, 2),
    "around a tile": ([127, 128, 129, 1, 2], [127, 128, 129, 1, 2], 2, 2),
    "around two tiles": ([255, 256, 257], [255, 256, 257], 3, 1),
    "long and short": ([700, 3, 64, 1024, 31], [700, 3, 64, 1024, 31], 2, 2),
    "groups of 4": ([200, 33, 1], [200, 33, 1], 8, 2),
    "groups of 3": ([130, 50, 85], [130, 50, 85], 6, 2),
    "groups of 5": ([77, 300], [77, 300], 5, 1),
    "groups of 7, chunks": ([40, 1, 19], [300, 129, 19], 14, 2),
    "one key head": ([100, 30], [100, 30], 16, 1),
    "chunks after a cache": ([64, 1, 130, 5], [512, 300, 131, 640], 4, 4),
    "queries without keys": ([200, 10, 140], [60, 0, 139], 2, 1),
    "sequences without rows": ([0, 50, 0, 0, 20, 0], [30, 50, 0, 7, 20, 0], 2, 2),
    "new tokens": ([1, 1, 1, 1, 1], [1, 64, 517, 2000, 33], 4, 4),
    "new tokens, groups": ([1, 1, 1], [3000, 129, 15], 16, 2),
    "few tokens, groups": ([2, 1, 2, 0], [640, 1, 1500, 5], 8, 1),
    "few tokens, empty rows": ([3, 2, 4], [1, 0, 900], 4, 1),
    "many heads to one": ([3, 2], [20, 150], 64, 1),
    "128 heads to one": ([2, 1], [9, 140], 128, 1),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("mode,hd", [(1, 64), (0, 64), (0, 16)], ids=["bf16", "fp32", "fp32hd16"])
def test_attention(torch_cuda, name, mode, hd):
    lq, lk, Hq, Hkv = CASES[name]
    c = Packed(torch_cuda, 11, lq, lk, Hq, Hkv, hd, mode, fused=lq == lk)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("hd", [8, 32])
def test_attention_fp32_head_sizes(torch_cuda, hd):
    c = Packed(torch_cuda, 12, [65, 17, 1], [65, 40, 33], 6, 2, hd, 0)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
def test_attention_many_sequences(torch_cuda, mode):
    r = np.random.default_rng(4)
    lk = [int(x) for x in np.exp(r.uniform(0, np.log(300), 150)).round()]
    lq = [int(r.integers(0, x + 2)) for x in lk]
    c = Packed(torch_cuda, 13, lq, lk, 4, 2, 64, mode)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (3, 3), (16, 4), (12, 12)])
def test_attention_few_queries_of_many_sequences(torch_cuda, Hq, Hkv):
    """New tokens over caches of every length from none on, some sequences without a query between them."""
    r = np.random.default_rng(7)
    lk = [int(x) for x in np.exp(r.uniform(0, np.log(900), 90)).round()] + [5000, 0, 0, 40, 16, 0, 2600]
    lq = [int(x) for x in r.integers(0, min(3, 16 // (Hq // Hkv)) + 1, len(lk))]
    lq[90], lq[96] = 0, 1  # a long cache that nobody asks for
    c = Packed(torch_cuda, 26, lq, lk, Hq, Hkv, 64, 1)
    c.forward()
    c.check(back=False)


def test_attention_few_queries_neighbours_do_not_leak(torch_cuda):
    """Caches of NaN and infinities between others, that end and begin inside a tile of keys."""
    torch = torch_cuda
    lk = [5, 9, 16, 200, 3, 1, 77, 31, 500]
    c = Packed(torch, 27, [1] * len(lk), lk, 8, 4, 64, 1)
    c.forward()
    o, lse = c.o.clone(), c.lse.clone()
    for s in range(0, len(lk), 2):
        at = slice(int(c.cu_k[s]), int(c.cu_k[s + 1]))
        c.tk[at], c.tv[at] = float("nan"), float("inf")
    c.forward()
    torch.cuda.synchronize()
    for s in range(1, len(lk), 2):
        row = int(c.cu_q[s])
        assert torch.equal(o[row], c.o[row]) and torch.equal(lse[:, row], c.lse[:, row]), s


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk", [([40, 0, 7], [0, 0, 0]), ([1, 1], [0, 0]), ([0, 0], [70, 300]), ([0, 0, 0], [0, 0, 0])])
def test_attention_batches_without_keys_or_queries(torch_cuda, mode, lq, lk):
    """Nothing to see (outputs 0, lse -inf, gradients 0), or nobody that sees: dK and dV are 0."""
    c = Packed(torch_cuda, 28, lq, lk, 4, 2, 64, mode, before=0, after=0)
    c.forward()
    c.backward()
    c.check()


def test_attention_no_queries_announced(torch_cuda):
    """max_q = 0 with queries there: reported, and nothing is written."""
    torch = torch_cuda
    c = Packed(torch, 29, [1, 1], [3000, 700], 4, 4, 64, 1)
    c.max_q = 0
    before = c.o.clone(), c.lse.clone()
    c.forward()
    torch.cuda.synchronize()
    assert c.status.item() == 8 and torch.equal(before[0], c.o) and torch.equal(before[1], c.lse)


@pytest.mark.parametrize("Hq,Hkv,lo,hi", [(12, 12, 1, 520), (8, 4, 20, 100), (25, 25, 100, 700)])
def test_attention_more_items_than_ctas(torch_cuda, Hq, Hkv, lo, hi):
    """Many short sequences: several work items for each CTA of the persistent kernels, runs of them with one tile."""
    r = np.random.default_rng(6)
    lk = [int(x) for x in r.integers(lo, hi, 40)]
    c = Packed(torch_cuda, 20, lk, lk, Hq, Hkv, 64, 1, fused=True)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
def test_attention_large_scores(torch_cuda, mode):
    """Scores up to about +-150: the running maximum moves far, most weights underflow."""
    c = Packed(torch_cuda, 14, [300, 90, 1], [300, 400, 700], 4, 2, 64, mode, scale=16.0)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("queries", [300, 1], ids=["prompt", "new token"])
def test_attention_rising_scores(torch_cuda, queries):
    """Every key block's scores exceed the one before by far (no block's maximum serves the next), then fall."""
    c = Packed(torch_cuda, 15, [queries], [1100], 2, 2, 64, 1)
    ramp = np.concatenate([np.linspace(0, 60, 700), np.linspace(60, -60, 400)])
    c.q[c.real_q] = 0
    c.q[c.real_q, :, 0] = 8.0
    c.k[c.real_k, :, 0] = data.round_to_bf16(ramp.astype(np.float32))[:, None]
    c.tq.copy_(dev(c.q.astype(np.float32)))
    c.tk.copy_(dev(c.k.astype(np.float32)))
    c.forward()
    c.check(back=False)


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
def test_attention_neighbours_do_not_leak(torch_cuda, mode):
    """A sequence of NaN and infinities between two others reaches neither of them, in any output."""
    torch = torch_cuda
    lq, lk = [70, 90, 33], [200, 90, 161]
    c = Packed(torch, 16, lq, lk, 4, 2, 64, mode)
    c.forward()
    c.backward()
    good = [x.clone() for x in (c.o, c.lse, c.dq, c.dk, c.dv)]
    a, b = (slice(int(x[1]), int(x[2])) for x in (c.cu_q, c.cu_k))
    for t, at in ((c.tq, a), (c.tk, b), (c.tv, b), (c.tdout, a)):
        t[at] = float("nan")
        t[at][::2] = float("inf")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    for x, y in zip((c.o, c.dq, c.dk, c.dv), (good[0], *good[2:])):
        at = a if x.shape[0] == c.rows_q and x.shape[1] == 4 else b
        x, y = x.clone(), y.clone()
        x[at] = 0
        y[at] = 0
        assert torch.equal(x, y)
    assert torch.equal(c.lse[:, :a.start], good[1][:, :a.start]) and torch.equal(c.lse[:, a.stop:], good[1][:, a.stop:])


@pytest.mark.parametrize("queries", [90, 1], ids=["prompt", "new token"])
def test_attention_bad_offsets_are_reported(torch_cuda, queries):
    """Offsets that descend, leave the buffers or exceed the given maximum set bit 8 and touch nothing outside."""
    torch = torch_cuda
    for cu_q, cu_k in (([0, 50, 20, 100], [0, 50, 60, 100]), ([0, 50, 60, 100], [0, 50, 20, 100]),
                       ([-5, 50, 60, 100], [0, 50, 60, 100]), ([0, 50, 60, 101], [0, 50, 60, 100]),
                       ([0, 50, 60, 100], [0, 50, 60, 1 << 30]), ([0, 0, 0, 0], [0, 95, 97, 100])):
        c = Packed(torch, 17, [50, 10, 40], [50, 10, 40], 4, 2, 64, 1, before=0, after=0)
        c.dev_cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu_q, cu_k)]
        c.max_q, c.max_k = queries, 90
        c.forward()
        torch.cuda.synchronize()
        assert c.status.item() == 8, (cu_q, cu_k)
        c.status.zero_()
        c.backward()
        torch.cuda.synchronize()
        assert c.status.item() == 8, (cu_q, cu_k)


@pytest.mark.parametrize("lq,lk", [([300, 41, 700], [300, 41, 700]), ([1, 1, 1], [300, 4100, 700])])
def test_attention_same_bits_again_on_a_stream_and_in_a_graph(torch_cuda, lq, lk):
    """The same bits on another stream, and from a captured graph that is replayed on changed inputs and offsets."""
    torch = torch_cuda
    c = Packed(torch, 18, lq, lk, 8, 2, 64, 1)
    names = ("o", "lse", "dq", "dk", "dv")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    first = {n: getattr(c, n).clone() for n in names}
    side = torch.cuda.Stream()
    for n in names:
        getattr(c, n).fill_(c.FILL)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep = [c.forward(stream=side), c.backward(stream=side)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(first[n], getattr(c, n)), n
    del keep
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward()
        c.backward()
    # other values and other (shorter) sequences, then the first ones again
    was = [t.clone() for t in (c.tq, *c.dev_cu)]
    c.tq.mul_(0.5)
    c.dev_cu[1][1:] -= 7
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first["o"], c.o)
    for t, w in zip((c.tq, *c.dev_cu), was):
        t.copy_(w)
    for n in names:
        getattr(c, n).fill_(c.FILL)
    graph.replay()
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(first[n], getattr(c, n)), n
    c.check()


def test_attention_graphs_that_share_their_workspaces(torch_cuda):
    """Graphs of one memory pool, replayed in turn: each call writes its lists and parts before it reads them."""
    torch = torch_cuda
    cs = [Packed(torch, 31, [300, 41, 700], [300, 41, 700], 8, 2, 64, 1), Packed(torch, 32, [1] * 5, [900, 1, 40, 3000, 0], 8, 2, 64, 1),
          Packed(torch, 33, [130, 64], [700, 64], 4, 4, 64, 1), Packed(torch, 34, [2, 1], [2000, 77], 12, 12, 64, 1)]
    names = ("o", "lse", "dq", "dk", "dv")
    first = []
    for c in cs:
        c.forward()
        c.backward()
        first.append([getattr(c, n).clone() for n in names])
    torch.cuda.synchronize()
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            c.forward()
            c.backward()
        graphs.append(g)
    for _ in range(2):
        for c in cs:
            for n in names:
                getattr(c, n).fill_(c.FILL)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for c, f in zip(cs, first):
            for n, x in zip(names, f):
                assert torch.equal(x, getattr(c, n)), n


def test_attention_equals_the_rectangular_one(torch_cuda):
    """Equal lengths and a key head per query head: the attention of the step, within both kernels' bounds."""
    torch = torch_cuda
    from step_gpt_train_gb300.gpt2 import gpt2_op_attention_forward
    B, T, H = 3, 384, 4
    c = Packed(torch, 19, [T] * B, [T] * B, H, H, 64, 1, before=0, after=0)
    c.forward()
    qkv = torch.cat([t.reshape(B * T, H * 64) for t in (c.tq, c.tk, c.tv)], 1)
    o, lse = torch.empty(B * T, H * 64, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, T, device="cuda")
    gpt2_op_attention_forward(o, lse, qkv, B, T, H)
    torch.cuda.synchronize()
    _, _, bo, bl = P.attention_forward(c.q, c.k, c.v, c.cu_q, c.cu_k, 1)
    within(host(c.o), host(o).reshape(B * T, H, 64), 2 * bo, "o")
    within(host(c.lse), host(lse).transpose(1, 0, 2).reshape(H, B * T), 2 * bl, "lse")


# ---------------------------------------------------------------- token log-probabilities

# fp32 sums of V terms in a tree or strided chains of at most V/128: each term's relative error is that of its
# exponential and of its argument, whose rounding is at most F32 * (|z| + |m|) (the shift) and F32 * |d| (log2 e)
def lp_bounds(z, V, ref):
    lse, logp, ent, _, top = ref
    m = np.where(np.isfinite(z[:, :V]), np.abs(z[:, :V]), 0).max(axis=1)
    es = P.F32 * (4 * m + V / 128 + 64)
    abslse = np.abs(np.where(np.isfinite(lse), lse, 0))
    bl = es + 4 * P.F32 * (1 + abslse)
    # entropy = log S - T/S: T's terms p |d| (at most log V + 1 in sum) carry the same relative errors
    be = 2 * es * (2 + np.log(V)) + 8 * P.F32 * (1 + np.log(V))
    return bl, bl + 2 * P.F32 * m + 2 * P.F32 * np.abs(np.where(np.isfinite(logp), logp, 0)), be


def run_logprobs(torch, z, t, V, k, mode, entropy=True):
    from step_gpt_train_gb300.gpt2 import gpt2_op_token_logprobs
    N = len(z)
    zt, tt = dev(z.astype(np.float32), mode), torch.from_numpy(t.astype(np.int32)).cuda()
    logp, lse, ent = (torch.full((N,), 7.0, device="cuda") for _ in range(3))
    top, ids = torch.full((N, k), 7.0, device="cuda"), torch.full((N, k), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gpt2_op_token_logprobs(logp, lse, ent if entropy else None, zt, tt, V, top_logp=top if k else None,
                           top_ids=ids if k else None, status=status)
    torch.cuda.synchronize()
    return zt, tt, logp, lse, ent, top, ids, status


def check_logprobs(torch, z, t, V, k, mode):
    zt, tt, logp, lse, ent, top, ids, status = run_logprobs(torch, z, t, V, k, mode)
    ref = P.token_logprobs(z, t, V, k)
    bl, bp, be = lp_bounds(z, V, ref)
    within(host(lse), ref[0], bl, "lse")
    within(host(logp), ref[1], bp, "logp")
    within(host(ent), ref[2], be, "entropy")
    assert (ids.cpu().numpy() == ref[3]).all()
    within(host(top), ref[4], np.repeat(bp[:, None] + 2 * P.F32 * np.abs(np.where(np.isfinite(ref[4]), ref[4], 0)).max(
        axis=1, initial=0)[:, None], k, 1), "top")
    assert status.item() == (4 if ((t < 0) | (t >= V)).any() else 0)
    assert torch.equal(zt, dev(z.astype(np.float32), mode)) or not np.isfinite(z).all()
    return zt, tt, lse, ent


def check_logprobs_backward(torch, z, t, V, mode, zt, tt, lse, ent, seed=5):
    from step_gpt_train_gb300.gpt2 import gpt2_op_token_logprobs_backward
    N, Vp = z.shape
    r = np.random.default_rng(seed)
    g, a, b = (r.standard_normal(N).astype(np.float32) for _ in range(3))
    gt, at, bt = (torch.from_numpy(x).cuda() for x in (g, a, b))
    none = np.zeros(N)
    for use in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        dz = torch.full_like(zt, 7.0)
        gpt2_op_token_logprobs_backward(dz, zt, tt if use[0] else None, lse, ent if use[2] else None, V,
                                        dlogp=gt if use[0] else None, dlse=at if use[1] else None,
                                        dentropy=bt if use[2] else None)
        ref, size = P.token_logprobs_backward(z, t, V, *(x if u else none for x, u in zip((g, a, b), use)))
        # p = exp(z - lse): lse's error and the argument's rounding; log p and the entropy enter with their errors
        refs = P.token_logprobs(z, t, V, 0)
        bl, bp, be = lp_bounds(z, V, refs)
        p = np.exp(np.where(np.isfinite(z[:, :V]), z[:, :V], -np.inf) - np.where(np.isfinite(refs[0]), refs[0], 0)[:, None])
        bound = (bp[:, None] + 16 * P.F32) * size * 2 + (P.BF16 if mode else 2 * P.F32) * np.abs(ref) + 1e-38
        bound[:, :V] += use[2] * np.abs(b)[:, None] * p * (bp + be)[:, None]
        # a gradient below the smallest normal number of fp32 may be flushed
        within(host(dz), ref, bound + 2.0 ** -126, f"dlogits {use}")
        assert (host(dz)[:, V:] == 0).all()
    same = zt.clone()
    gpt2_op_token_logprobs_backward(same, same, tt, lse, ent, V, dlogp=gt, dentropy=bt)
    torch.cuda.synchronize()
    assert torch.equal(same, dz)  # in place, and again: the same bits


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,V,Vp,k", [(1, 1, 8, 1), (3, 7, 8, 7), (5, 64, 64, 64), (4, 300, 304, 5), (257, 512, 512, 3), (5, 503, 512, 32), (7, 477, 480, 64),
                                      (9, 4097, 4104, 33), (6, 50257, 50304, 20), (3, 50257, 50304, 0),
                                      (2, 130001, 130048, 64), (1, 300001, 300008, 8)])
def test_logprobs(torch_cuda, N, V, Vp, k, mode):
    r = np.random.default_rng(N + V)
    z = inputs(21, (N, Vp), 3.0, mode).astype(np.float64)
    z[:, V:] = 1e4  # padding columns count for nothing
    t = r.integers(0, V, N)
    zt, tt, lse, ent = check_logprobs(torch_cuda, z, t, V, k, mode)
    check_logprobs_backward(torch_cuda, z, t, V, mode, zt, tt, lse, ent)


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [1000, 50257])
def test_logprobs_ties_and_special_rows(torch_cuda, V, mode):
    Vp = -(-V // 8) * 8
    z = inputs(22, (12, Vp), 2.0, mode).astype(np.float64)
    z[0] = 0.0                       # all equal: the first columns, entropy log V
    z[1] = np.tile([0.0, -0.0], Vp // 2)  # the zeros are equal
    z[2] = -np.inf                   # no distribution
    z[3] = -np.inf
    z[3, V - 1] = 2.0                # one token has all of it
    z[4, ::2] = -np.inf              # masked tokens
    z[5] = np.round(z[5])            # few values, many ties
    z[6] = np.linspace(-20, 20, Vp)  # rising: every column a new largest
    z[7] = np.linspace(20, -20, Vp)
    z[8] = -1e30                     # masks of a very low value
    z[8, 17] = 1.0
    z[9] += 3e4                      # far from zero
    z[10] = np.where(np.arange(Vp) % 256 == 3, 50.0, -50.0)  # the large ones in one residue class
    z[11, :4] = [1e4, 1e4, -1e4, 9e3]
    z = data.round_to_bf16(z.astype(np.float32)).astype(np.float64) if mode == 1 else z.astype(np.float32).astype(np.float64)
    t = np.array([V - 1, 3, 0, V - 1, 1, 0, V - 1, 0, 17, 5, -1, V])
    z[:, V:] = np.nan                # padding columns are not looked at
    zt, tt, lse, ent = check_logprobs(torch_cuda, z, t, V, 40, mode)
    check_logprobs_backward(torch_cuda, z, t, V, mode, zt, tt, lse, ent)


def test_logprobs_non_finite_rows(torch_cuda):
    """A NaN or +inf makes its own row's results what the formulas give; ids stay in range; other rows are as ever."""
    torch = torch_cuda
    V = 50257
    z = inputs(23, (4, 50304), 2.0, 1).astype(np.float64)
    t = np.array([1, 2, 3, 4])
    plain = run_logprobs(torch, z, t, V, 9, 1)
    z[1, 40000], z[2, 777] = np.nan, np.inf
    got = run_logprobs(torch, z, t, V, 9, 1)
    _, _, logp, lse, ent, top, ids, _ = got
    assert torch.isnan(lse[1]) and torch.isnan(logp[1]) and torch.isnan(ent[1]) and torch.isnan(top[1]).all()
    assert lse[2].item() == np.inf and logp[2].item() == -np.inf and torch.isnan(ent[2]) and ids[2, 0].item() == 777
    assert ((ids >= 0) & (ids < V)).all()
    for a, b in zip(got[2:7], plain[2:7]):
        assert torch.equal(a[[0, 3]], b[[0, 3]])


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,k", [(40, 40), (477, 32), (503, 64), (1000, 20), (1000, 64), (50257, 5), (50257, 20)])
def test_logprobs_alternatives_of_many_rows(torch_cuda, V, k, mode):
    """More rows than four blocks on each SM, ties and masks among them."""
    Vp, N = -(-V // 8) * 8 + 8, 700
    z = inputs(24, (N, Vp), 2.0, mode).astype(np.float64)
    z[1::9] = 0.0
    z[2::9] = np.round(z[2::9])
    z[3::9] = -np.inf
    z[12::9, V // 2] = 1.0           # (row 3 stays without any token)
    z[4::9, ::2] = -np.inf
    z[5::9] = np.linspace(-20, 20, Vp).astype(np.float32)
    z[6::9] = -1e30
    z[6::9, 17] = 1.0
    z = data.round_to_bf16(z.astype(np.float32)).astype(np.float64) if mode == 1 else z.astype(np.float32).astype(np.float64)
    z[:, V:] = np.nan                # padding columns are not looked at
    check_logprobs(torch_cuda, z, np.random.default_rng(5).integers(0, V, N), V, k, mode)


@pytest.mark.parametrize("N", [3, 400, 700])
def test_logprobs_rows_of_nan(torch_cuda, N):
    """Rows of NaN, with more of them than the alternatives asked for: ids are the first such columns."""
    torch = torch_cuda
    V, k = 50257, 9
    z = inputs(25, (N, 50304), 2.0, 1).astype(np.float64)
    t = np.full(N, 4)
    plain = run_logprobs(torch, z, t, V, k, 1)
    z[1], z[N - 1, 300:] = np.nan, np.nan
    z[1, ::2] *= -1                  # of either sign
    got = run_logprobs(torch, z, t, V, k, 1)
    ids = got[6].cpu().numpy()
    assert (ids[1] == np.arange(k)).all() and (ids[N - 1] == 300 + np.arange(k)).all()
    for a, b in zip(got[2:7], plain[2:7]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2:N - 1], b[2:N - 1])


def test_logprobs_many_rows_stream_and_graph(torch_cuda):
    torch = torch_cuda
    from step_gpt_train_gb300.gpt2 import gpt2_op_token_logprobs, gpt2_op_token_logprobs_backward
    N, V, Vp, k = 1500, 5003, 5008, 7
    z = torch.randn(N, Vp, device="cuda").bfloat16()
    t = torch.randint(0, V, (N,), dtype=torch.int32, device="cuda")
    out = [torch.zeros(N, device="cuda") for _ in range(3)] + [torch.zeros(N, k, device="cuda"),
                                                               torch.zeros(N, k, dtype=torch.int32, device="cuda")]
    dz, g = torch.zeros_like(z), torch.randn(N, device="cuda")

    def both(stream=None):
        gpt2_op_token_logprobs(out[0], out[1], out[2], z, t, V, out[3], out[4], stream=stream)
        gpt2_op_token_logprobs_backward(dz, z, t, out[1], out[2], V, dlogp=g, dentropy=g, stream=stream)
    both()
    first = [x.clone() for x in (*out, dz)]
    ref = P.token_logprobs(host(z), t.cpu().numpy(), V, k)
    assert (out[4].cpu().numpy() == ref[3]).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for x in (*out, dz):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (*out, dz)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- offsets past 32 bits

@pytest.mark.parametrize("lq,lk", [([700, 1, 1500], [700, 1, 1500]), ([2, 0, 1], [700, 1, 1500])])
def test_attention_rows_far_apart(torch_cuda, lq, lk):
    """Buffers of more than 2^31 elements (a row stride of 2^20): the same bits as from rows side by side."""
    torch = torch_cuda
    stride = 1 << 20
    c = Packed(torch, 30, lq, lk, 4, 2, 64, 1, before=0, after=0)
    c.forward()
    c.backward()
    near = [x.clone() for x in (c.o, c.lse, c.dq, c.dk, c.dv)]
    wide = torch.empty(c.rows_k * stride, dtype=torch.bfloat16, device="cuda")
    at = [0]

    def far(t):  # its own columns of the wide rows
        x = wide.as_strided((t.shape[0], t.shape[1], 64), (stride, 64, 1), at[0])
        at[0] += t.shape[1] * 64
        x.copy_(t)
        return x
    for name in ("tq", "tk", "tv", "tdout", "o", "dq", "dk", "dv"):
        setattr(c, name, far(getattr(c, name)))
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    for x, y in zip(near, (c.o, c.lse, c.dq, c.dk, c.dv)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("k", [0, 6])
def test_logprobs_more_logits_than_32_bits_count(torch_cuda, k):
    torch = torch_cuda
    from step_gpt_train_gb300.gpt2 import gpt2_op_token_logprobs, gpt2_op_token_logprobs_backward
    N, n, V, Vp = 43000, 700, 50257, 50304

    def run(z, dz):
        rows = len(z)
        t = torch.full((rows,), 50256, dtype=torch.int32, device="cuda")
        out = [torch.zeros(rows, device="cuda") for _ in range(3)]
        top = [torch.zeros(rows, k, device="cuda"), torch.zeros(rows, k, dtype=torch.int32, device="cuda")] if k else [None] * 2
        gpt2_op_token_logprobs(*out, z, t, V, *top)
        gpt2_op_token_logprobs_backward(dz, z, t, out[1], out[2], V, dlogp=out[0], dentropy=out[2])
        return [x[-n:].clone() for x in (*out, *top, dz) if x is not None]
    some = torch.randn(n, Vp, device="cuda").bfloat16()
    z = torch.zeros(N, Vp, dtype=torch.bfloat16, device="cuda")
    z[-n:] = some
    few = run(some, torch.empty_like(some))
    for x, y in zip(run(z, z), few):  # the gradient in place
        assert torch.equal(x, y)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
def test_scoring_a_packed_batch(torch_cuda, mode):
    """Packed documents through a projection, attention, an output head and the log-probabilities, and the gradient of
    a weighted sum of log-probabilities and entropies back to the hidden states: every op of the run on its own
    inputs against the formula, and the whole against central differences along one direction (fp32)."""
    torch = torch_cuda
    from step_gpt_train_gb300 import gpt2 as G
    Hq, Hkv, hd, C, V, Vp = 4, 2, 64, 256, 200, 208
    lens = [50, 1, 130, 7]
    T = sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x, wqkv, wout = (inputs(s, shape, std, mode) for s, shape, std in ((31, (T, C), 1.0), (32, ((Hq + 2 * Hkv) * hd, C), 0.06),
                                                                     (33, (Vp, C), 0.1)))
    t = torch.from_numpy(np.random.default_rng(0).integers(0, V, T).astype(np.int32)).cuda()
    g, b = (torch.from_numpy(inputs(s, (T,), 0.1, 0)).cuda() for s in (34, 35))
    w1, w2 = dev(wqkv, mode), dev(wout, mode)
    new = lambda *s: torch.empty(*s, dtype=w1.dtype, device="cuda")  # noqa: E731
    heads = lambda y: (y[:, :Hq * hd].unflatten(1, (Hq, hd)), y[:, Hq * hd:(Hq + Hkv) * hd].unflatten(1, (Hkv, hd)),  # noqa: E731
                       y[:, (Hq + Hkv) * hd:].unflatten(1, (Hkv, hd)))

    def forward(xt):
        qkv, o, z = new(T, w1.shape[0]), new(T, Hq, hd), new(T, Vp)
        lse_a, logp, lse, ent = torch.empty(Hq, T, device="cuda"), *(torch.empty(T, device="cuda") for _ in range(3))
        G.gpt2_op_matmul(qkv, xt, 0, w1, 0, T, w1.shape[0], C)
        G.gpt2_op_attention_packed_forward(o, lse_a, *heads(qkv), cu, cu, max(lens), max(lens))
        G.gpt2_op_matmul(z, o, 0, w2, 0, T, Vp, C)
        G.gpt2_op_token_logprobs(logp, lse, ent, z, t, V)
        return qkv, o, z, lse_a, logp, lse, ent

    def loss(xt):
        *_, logp, _, ent = forward(xt)
        return (logp.double() * g + ent.double() * b).sum().item()

    xt = dev(x, mode)
    qkv, o, z, lse_a, logp, lse, ent = forward(xt)
    dz, do, dqkv, dx = new(T, Vp), new(T, Hq, hd), new(T, w1.shape[0]), new(T, C)
    G.gpt2_op_token_logprobs_backward(dz, z, t, lse, ent, V, dlogp=g, dentropy=b)
    G.gpt2_op_matmul(do, dz, 0, w2, 1, T, C, Vp)
    G.gpt2_op_attention_packed_backward(*heads(dqkv), do, *heads(qkv), o, lse_a, cu, cu, max(lens), max(lens))
    G.gpt2_op_matmul(dx, dqkv, 0, w1, 1, T, C, w1.shape[0])
    torch.cuda.synchronize()
    q, k, v = (host(y) for y in heads(qkv))
    cun = cu.cpu().numpy()
    ro, rl, bo, bl = P.attention_forward(q, k, v, cun, cun, mode)
    within(host(o), ro, bo, "o")
    within(host(lse_a), rl, bl, "lse")
    refs = P.attention_backward(host(do), q, k, v, cun, cun, mode)
    for y, r, bd in zip(heads(dqkv), refs[:3], refs[3:]):
        within(host(y), r, bd, "dqkv")
    ref = P.token_logprobs(host(z), t.cpu().numpy(), V, 0)
    bl, bp, be = lp_bounds(host(z), V, ref)
    within(host(logp), ref[1], bp, "logp")
    within(host(ent), ref[2], be, "entropy")
    if mode == 0:
        # each evaluation of the loss carries T terms' fp32 errors (below 1e-6 each, adding in quadrature to below
        # 1e-5): over 2h = 0.02 that is 1e-3, and the third derivative's h^2 term is of the same size; |dx| |d| is of order 1
        d = torch.from_numpy(inputs(36, (T, C), 1.0, 0)).cuda()
        d /= d.norm()
        h = 1e-2
        by_diff = (loss(xt + h * d) - loss(xt - h * d)) / (2 * h)
        want = (dx.double() * d).sum().item()
        assert abs(by_diff - want) <= 4e-3 + 1e-2 * abs(want), (by_diff, want)
