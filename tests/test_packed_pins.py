"""Pins of the oracle's packed attention and token log-probabilities (CPU), and
the refusals of their entry points, which touch no device."""
import math

import numpy as np
import pytest

from oracle import packed_ref as P


def _attention_case(seed, lq, lk, Hq, Hkv, hd):
    r = np.random.default_rng(seed)
    cu_q, cu_k = np.concatenate([[0], np.cumsum(lq)]), np.concatenate([[0], np.cumsum(lk)])
    q = r.standard_normal((cu_q[-1], Hq, hd))
    k, v = (r.standard_normal((cu_k[-1], Hkv, hd)) for _ in range(2))
    return q, k, v, r.standard_normal(q.shape), cu_q, cu_k


@pytest.mark.parametrize("lq,lk,Hq,Hkv", [([5, 1, 9], [5, 1, 9], 4, 2), ([3, 2], [7, 2], 6, 1), ([1, 1], [4, 11], 2, 2)])
def test_attention_is_torch_sdpa_and_its_autograd(lq, lk, Hq, Hkv):
    import torch
    import torch.nn.functional as F
    q, k, v, dout, cu_q, cu_k = _attention_case(0, lq, lk, Hq, Hkv, 8)
    o, lse, _, _ = P.attention_forward(q, k, v, cu_q, cu_k, 0)
    grads = P.attention_backward(dout, q, k, v, cu_q, cu_k, 0)[:3]
    for a, b in P.sequences(cu_q, cu_k):
        tq, tk, tv = (torch.from_numpy(np.ascontiguousarray(x)).requires_grad_() for x in (q[a], k[b], v[b]))
        nq, nk = len(q[a]), len(k[b])
        mask = torch.ones(nq, nk, dtype=torch.bool).tril(nk - nq)
        rep = lambda t: t.repeat_interleave(Hq // Hkv, 1).transpose(0, 1)  # noqa: E731
        y = F.scaled_dot_product_attention(tq.transpose(0, 1), rep(tk), rep(tv), attn_mask=mask).transpose(0, 1)
        np.testing.assert_allclose(o[a], y.detach().numpy(), rtol=1e-12, atol=1e-12)
        y.backward(torch.from_numpy(np.ascontiguousarray(dout[a])))
        for g, t, at in zip(grads, (tq, tk, tv), (a, b, b)):
            np.testing.assert_allclose(g[at], t.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_attention_rows_without_keys_and_sequences_without_rows():
    q, k, v, dout, cu_q, cu_k = _attention_case(1, [4, 0, 3], [2, 3, 0], 2, 1, 8)
    o, lse, _, _ = P.attention_forward(q, k, v, cu_q, cu_k, 0)
    assert (o[:2] == 0).all() and np.isneginf(lse[:, :2]).all() and np.isfinite(lse[:, 2:4]).all()
    assert (o[4:] == 0).all() and np.isneginf(lse[:, 4:]).all()
    dq, dk, dv = P.attention_backward(dout, q, k, v, cu_q, cu_k, 0)[:3]
    assert (dq[:2] == 0).all() and (dq[4:] == 0).all() and (dk[2:] == 0).all() and (dv[2:] == 0).all()


def test_attention_backward_by_differences():
    q, k, v, dout, cu_q, cu_k = _attention_case(2, [3, 2], [4, 2], 4, 2, 8)
    f = lambda: (P.attention_forward(q, k, v, cu_q, cu_k, 0)[0] * dout).sum()  # noqa: E731
    for x, g in zip((q, k, v), P.attention_backward(dout, q, k, v, cu_q, cu_k, 0)[:3]):
        for i in np.ndindex(*x.shape):
            at, h = x[i], 1e-5
            x[i] = at + h
            up = f()
            x[i] = at - h
            down = f()
            x[i] = at
            assert abs((up - down) / (2 * h) - g[i]) < 1e-8


def test_token_logprobs_is_log_softmax_and_its_autograd():
    import torch
    r = np.random.default_rng(3)
    N, V, Vp, k = 6, 29, 32, 5
    z, t = r.standard_normal((N, Vp)) * 3, r.integers(0, V, N)
    lse, logp, ent, ids, top = P.token_logprobs(z, t, V, k)
    x = torch.from_numpy(z).requires_grad_()
    lp = torch.log_softmax(x[:, :V], 1)
    h = -(lp.exp() * lp).sum(1)
    np.testing.assert_allclose(logp, lp.detach().numpy()[np.arange(N), t], rtol=1e-13)
    np.testing.assert_allclose(ent, h.detach().numpy(), rtol=1e-12)
    want = torch.topk(lp, k, dim=1)
    assert (ids == want.indices.numpy()).all()
    np.testing.assert_allclose(top, want.values.detach().numpy(), rtol=1e-13)
    g, a, b = (r.standard_normal(N) for _ in range(3))
    loss = (lp[torch.arange(N), torch.from_numpy(t)] * torch.from_numpy(g)).sum() + \
        (torch.logsumexp(x[:, :V], 1) * torch.from_numpy(a)).sum() + (h * torch.from_numpy(b)).sum()
    loss.backward()
    np.testing.assert_allclose(P.token_logprobs_backward(z, t, V, g, a, b)[0], x.grad.numpy(), rtol=1e-9, atol=1e-13)


def test_token_logprobs_special_rows():
    V = 4
    z = np.array([[-np.inf] * 4, [0.0, -np.inf, -np.inf, -np.inf], [1.0, 2.0, 2.0, -0.0]])
    lse, logp, ent, ids, top = P.token_logprobs(z, np.array([1, 0, 2]), V, 3)
    assert np.isneginf(lse[0]) and np.isneginf(logp[0]) and ent[0] == 0 and np.isneginf(top[0]).all()
    assert lse[1] == 0 and logp[1] == 0 and ent[1] == 0
    assert ids[0].tolist() == [0, 1, 2] and ids[1].tolist() == [0, 1, 2] and ids[2].tolist() == [1, 2, 0]
    g, _ = P.token_logprobs_backward(z, np.array([1, 0, 2]), V, np.ones(3), np.ones(3), np.ones(3))
    assert (g[0] == 0).all() and np.isfinite(g).all()
    u = np.zeros((1, 50257))
    assert math.isclose(P.token_logprobs(u, np.array([0]), 50257, 0)[2][0], math.log(50257), rel_tol=1e-12)


# ---------------------------------------------------------------- refusals (nothing is launched)

@pytest.fixture(scope="module")
def lib():
    from step_gpt_train_gb300 import gpt2 as g
    return g.load_library(build=True)


ARG, WORKSPACE, OK = -1, -7, 0
A = 1 << 20  # an aligned address that no refused call touches


def forward(lib, **kw):
    c = dict(dtype=1, o=A, os=768, lse=A, q=A, qs=2304, k=A, ks=2304, v=A, vs=2304, cq=A, ck=A, n=3, tq=300, tk=300,
             mq=128, mk=128, hq=12, hkv=12, hd=64, sc=A, nb=1 << 40)
    c.update(kw)
    return lib.gpt2_op_attention_packed_forward(c["dtype"], c["o"], c["os"], c["lse"], c["q"], c["qs"], c["k"], c["ks"],
                                                c["v"], c["vs"], c["cq"], c["ck"], c["n"], c["tq"], c["tk"], c["mq"],
                                                c["mk"], c["hq"], c["hkv"], c["hd"], c["sc"], c["nb"], None, None)


def backward(lib, **kw):
    c = dict(dtype=1, dq=A, dqs=768, dk=A, dks=768, dv=A, dvs=768, do=A, dos=768, q=A, qs=768, k=A, ks=768, v=A, vs=768,
             o=A, os=768, lse=A, cq=A, ck=A, n=3, tq=300, tk=300, mq=128, mk=128, hq=12, hkv=12, hd=64, sc=A,
             nb=1 << 40)
    c.update(kw)
    return lib.gpt2_op_attention_packed_backward(*list(c.values()), None, None)


BAD = [dict(dtype=2), dict(n=-1), dict(tq=-1), dict(tk=-1), dict(mq=-1), dict(mk=-1), dict(hq=0), dict(hkv=0),
       dict(hkv=5), dict(hq=129 * 2, hkv=2), dict(hd=32), dict(hd=128), dict(dtype=0, hd=48), dict(q=None),
       dict(k=None), dict(v=None), dict(o=None), dict(lse=None), dict(cq=None), dict(ck=None), dict(q=A + 8),
       dict(k=A + 2), dict(v=A + 4), dict(o=A + 8), dict(qs=760), dict(ks=764), dict(vs=8), dict(os=700),
       dict(qs=1 << 31), dict(tq=(1 << 31) - 1), dict(tk=(1 << 31) - 1)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: ",".join(f"{k}={v}" for k, v in b.items()))
def test_attention_refusals(lib, bad):
    assert forward(lib, **bad) == ARG
    assert backward(lib, **bad) == ARG


@pytest.mark.parametrize("bad", [dict(dq=None), dict(dk=None), dict(dv=None), dict(do=None), dict(dq=A + 8),
                                 dict(dk=A + 2), dict(dv=A + 4), dict(do=A + 8), dict(dqs=760), dict(dks=764),
                                 dict(dvs=8), dict(dos=700)], ids=str)
def test_attention_backward_refusals(lib, bad):
    assert backward(lib, **bad) == ARG


def test_attention_workspace_and_nothing_to_do(lib):
    assert backward(lib, nb=lib.gpt2_op_attention_packed_backward_scratch(1, 3, 300, 300, 12, 12, 64) - 1) == WORKSPACE
    assert backward(lib, sc=None) == WORKSPACE
    need = lib.gpt2_op_attention_packed_forward_scratch(1, 3, 3, 1 << 17, 1, 1 << 17, 12, 12, 64)
    assert need > 0
    assert forward(lib, tq=3, tk=1 << 17, mq=1, mk=1 << 17, nb=need - 1) == WORKSPACE
    assert forward(lib, tq=3, tk=1 << 17, mq=1, mk=1 << 17, sc=None) == WORKSPACE
    for kw in (dict(n=0), dict(tq=0)):
        assert forward(lib, **kw) == OK
    assert backward(lib, n=0) == OK and backward(lib, tq=0, tk=0) == OK
    assert lib.gpt2_op_attention_packed_forward_scratch(1, -1, 1, 1, 1, 1, 12, 12, 64) == 0


def logprobs(lib, **kw):
    c = dict(dtype=1, logp=A, lse=A, ent=A, tl=A, ti=A, k=5, z=A, t=A, N=4, V=50257, Vp=50304)
    c.update(kw)
    return lib.gpt2_op_token_logprobs(*list(c.values()), None, None)


def logprobs_backward(lib, **kw):
    c = dict(dtype=1, dz=A, z=A, t=A, lse=A, ent=A, dlogp=A, dlse=A, dent=A, N=4, V=50257, Vp=50304)
    c.update(kw)
    return lib.gpt2_op_token_logprobs_backward(*list(c.values()), None, None)


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(N=-1), dict(V=0), dict(Vp=50256), dict(Vp=50257), dict(z=None),
                                 dict(z=A + 8), dict(lse=None)], ids=str)
def test_logprobs_refusals(lib, bad):
    assert logprobs(lib, **bad) == ARG
    assert logprobs_backward(lib, **bad) == ARG


def test_logprobs_more_refusals(lib):
    for bad in (dict(k=-1), dict(k=65), dict(k=5, V=4, Vp=8), dict(tl=None), dict(ti=None), dict(t=None),
                dict(logp=None)):
        assert logprobs(lib, **bad) == ARG, bad
    for bad in (dict(dz=None), dict(dz=A + 8), dict(t=None), dict(ent=None)):
        assert logprobs_backward(lib, **bad) == ARG, bad
    assert logprobs(lib, N=0) == OK and logprobs_backward(lib, N=0) == OK


def test_wrapper_refuses_operands_that_differ(lib):
    import torch
    from step_gpt_train_gb300 import gpt2 as g
    bf = torch.bfloat16
    q, k, cu, lse = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(9, 1, 64, dtype=bf), torch.tensor([0, 4]).int(), torch.zeros(2, 4)
    long = torch.tensor([0, 4])
    for o, ls, kk, v, cq, ck in ((q[:3], lse, k, k, cu, cu), (q.float(), lse, k, k, cu, cu), (q, lse[:1], k, k, cu, cu),
                                 (q, lse, k, k[:8], cu, cu), (q, lse, k.float(), k.float(), cu, cu),
                                 (q, lse, k, k, long, long), (q, lse, k, k, cu, torch.zeros(3).int())):
        with pytest.raises(ValueError):
            g.gpt2_op_attention_packed_forward(o, ls, q, kk, v, cq, ck, 4, 9)
        with pytest.raises(ValueError):
            g.gpt2_op_attention_packed_backward(q, k, k, q, q, kk, v, o, ls, cq, ck, 4, 9)
    with pytest.raises(ValueError):
        g.gpt2_op_attention_packed_backward(q[:2], k, k, q, q, k, k, q, lse, cu, cu, 4, 9)
    z, t, s = torch.zeros(4, 64, dtype=bf), torch.zeros(4).int(), torch.zeros(4)
    for bad in (z[:, :32], z[0], z.T):
        with pytest.raises(ValueError):
            g.gpt2_op_token_logprobs(s, s, s, bad, t, 30)
        with pytest.raises(ValueError):
            g.gpt2_op_token_logprobs_backward(z, bad, t, s, s, 30, dlogp=s)
        with pytest.raises(ValueError):
            g.gpt2_op_token_logprobs_backward(bad, z, t, s, s, 30, dlogp=s)
    with pytest.raises(ValueError):
        g.gpt2_op_token_logprobs(s, s, s, z, t, 30, top_logp=torch.zeros(4, 3))


def test_wrapper_refuses_other_layouts():
    import torch
    from step_gpt_train_gb300 import gpt2 as g
    x = torch.zeros(4, 2, 8)
    assert g._rows("x", x) == [16]
    assert g._rows("x", x, torch.zeros(4, 48)[:, 16:32].unflatten(1, (2, 8))) == [16, 48]
    assert g._rows("x", torch.zeros(1, 2, 8).expand(1, 2, 8)) == [16]
    for bad in (torch.zeros(4, 16), x.transpose(0, 1), x.transpose(1, 2), torch.zeros(4, 2, 16)[:, :, ::2]):
        with pytest.raises(ValueError):
            g._rows("x", bad)
        with pytest.raises(ValueError):
            g._rows("x", x, bad)
