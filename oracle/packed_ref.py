"""Plain numpy (float64) attention over packed sequences and token
log-probabilities, with the error bounds their tests use.

Shares no code with csrc/. Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8   # half a step of bf16, relative
F32 = 2.0 ** -24   # half a step of fp32, relative


def sequences(cu_q, cu_k):
    for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        yield slice(int(a), int(b)), slice(int(c), int(d))


def _scores(q, k):
    """Scaled scores of one head, -inf where query i may not see key j (j > i + lk - lq), and the sum of
    |q| |k| the rounding of a score is bounded by."""
    lq, lk = len(q), len(k)
    scale = 1.0 / np.sqrt(q.shape[1])
    hidden = np.arange(lk)[None, :] > np.arange(lq)[:, None] + lk - lq
    s = np.where(hidden, -np.inf, (q @ k.T) * scale)
    return s, np.where(hidden, 0.0, (np.abs(q) @ np.abs(k).T) * scale)


def _softmax(s):
    m = s.max(axis=1, keepdims=True, initial=-np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - m)
    l = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return e / np.where(l > 0, l, 1.0), lse


def attention_forward(q, k, v, cu_q, cu_k, mode):
    """o [Tq,Hq,hd], lse [Hq,Tq] and how far a kernel may be from them (same shapes). NaN marks rows of no
    sequence. mode 1: q, k, v are bf16 values, P is rounded to bf16 before P v, o on the way out; mode 0: fp32."""
    Tq, Hq, hd = q.shape
    group = Hq // k.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full((Hq, Tq), np.nan)
    do, dl = np.full(q.shape, np.nan), np.full((Hq, Tq), np.nan)
    for a, b in sequences(cu_q, cu_k):
        for h in range(Hq):
            kh, vh = k[b, h // group], v[b, h // group]
            s, sab = _scores(q[a, h], kh)
            p, lse[h, a] = _softmax(s)
            o[a, h] = p @ vh
            # a score is a sum of hd products: (hd + 4) roundings of at most the sum of |q||k|; exp turns a score's
            # absolute error into a relative one of p (and the exponential, its argument and the sums round too)
            es = (hd + 4) * F32 * sab.max(axis=1, initial=0.0) + (len(kh) + 16) * F32
            A = p @ np.abs(vh)
            rel = 2 * es + (len(kh) + 8) * F32
            out = BF16 if mode else 2 * F32
            do[a, h] = out * np.abs(o[a, h]) + (rel[:, None] + (BF16 if mode else 0.0)) * A * (1 + 2.0 ** -6) + 1e-30
            dl[h, a] = es + 4 * F32 * (1 + np.abs(np.where(np.isfinite(lse[h, a]), lse[h, a], 0.0)))
    return o, lse, do, dl


def attention_backward(dout, q, k, v, cu_q, cu_k, mode):
    """dq, dk, dv and how far a kernel may be from them. mode 1: the forward's o is rounded to bf16 (which moves
    D = rowsum(dO O)), P and dS are rounded to bf16 before their products, the gradients on the way out."""
    Tq, Hq, hd = q.shape
    Tk, Hkv, _ = k.shape
    group = Hq // Hkv
    dq, bq = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    dk, bk = np.full(k.shape, np.nan), np.full(k.shape, np.nan)
    dv, bv = np.full(k.shape, np.nan), np.full(k.shape, np.nan)
    u = BF16 if mode else 0.0
    out = BF16 if mode else 2 * F32
    scale = 1.0 / np.sqrt(hd)
    for a, b in sequences(cu_q, cu_k):
        for t in (dk, bk, dv, bv):
            t[b] = 0.0
        for h in range(Hq):
            kh, vh, qh, dy = k[b, h // group], v[b, h // group], q[a, h], dout[a, h]
            s, sab = _scores(qh, kh)
            p, lse = _softmax(s)
            n = len(kh) + len(qh) + 16
            # P from the scores and the stored lse: both off by their rounding
            lab = np.abs(np.where(np.isfinite(lse), lse, 0.0))
            es = (hd + 4) * F32 * sab.max(axis=1, initial=0.0) + n * F32 + 4 * F32 * (1 + lab)
            rel = (2 * es + n * F32)[:, None]
            o = p @ vh
            dp = dy @ vh.T
            D = (dy * o).sum(axis=1, keepdims=True)
            dpa = np.abs(dy) @ np.abs(vh).T
            eD = (u + out + rel) * (np.abs(dy) * (p @ np.abs(vh))).sum(axis=1, keepdims=True)
            ds = p * (dp - D)
            # dS: P's own error and rounding, dP's sum of hd products, D's error
            eds = (u + rel) * np.abs(ds) + p * ((hd + 4) * F32 * dpa + eD)
            dq[a, h] = scale * ds @ kh
            bq[a, h] = out * np.abs(dq[a, h]) + scale * (eds + n * F32 * np.abs(ds)) @ np.abs(kh)
            dv[b, h // group] += p.T @ dy
            bv[b, h // group] += ((u + rel + n * F32) * p).T @ np.abs(dy)
            dk[b, h // group] += scale * ds.T @ qh
            bk[b, h // group] += scale * (eds + n * F32 * np.abs(ds)).T @ np.abs(qh)
        for g, e in ((dk, bk), (dv, bv)):
            e[b] += out * np.abs(g[b]) + 1e-30
        bq[a] += 1e-30
    slack = 1 + 2.0 ** -6  # products of the first-order terms
    return dq, dk, dv, bq * slack, bk * slack, bv * slack


def token_logprobs(z, targets, V, k):
    """lse, logp, entropy, top ids, top log-probabilities of the rows of z [N, >= V]."""
    z = z[:, :V]
    m = z.max(axis=1, keepdims=True)
    some = np.isfinite(m[:, 0])
    z0 = np.where(some[:, None], z, 0.0)
    m0 = np.where(some[:, None], m, 0.0)
    e = np.exp(z0 - m0)
    lse = np.where(some, (m0 + np.log(e.sum(axis=1, keepdims=True)))[:, 0], -np.inf)
    lp = np.where(some[:, None], z0 - np.where(some, lse, 0.0)[:, None], -np.inf)
    p = np.exp(lp)
    ent = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(axis=1)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    t = np.where((targets < 0) | (targets >= V), 0, targets)
    return lse, lp[np.arange(len(z)), t], ent, ids, np.take_along_axis(lp, ids, axis=1)


def token_logprobs_backward(z, targets, V, dlogp, dlse, dent):
    """dlogits [N, Vp], and the sum of the absolute values of its terms."""
    N, Vp = z.shape
    lse, _, ent, _, _ = token_logprobs(z, targets, V, 0)
    some = np.isfinite(lse)
    lp = np.where(some[:, None], z[:, :V] - np.where(some, lse, 0.0)[:, None], -np.inf)
    p = np.exp(lp)
    lp0 = np.where(p > 0, lp, 0.0)
    g = np.zeros((N, Vp))
    g[:, :V] = p * (dlse - dlogp)[:, None] - dent[:, None] * p * (lp0 + ent[:, None])
    size = np.zeros((N, Vp))
    size[:, :V] = p * ((np.abs(dlse) + np.abs(dlogp))[:, None] + np.abs(dent)[:, None] * (np.abs(lp0) + ent[:, None]))
    t = np.where((targets < 0) | (targets >= V), 0, targets)
    r = np.arange(N)
    g[r, t] += np.where(some, dlogp, 0.0)
    size[r, t] += np.where(some, np.abs(dlogp), 0.0)
    return g, size
