"""Cases of the packed-sequence attention and the token log-probabilities, with their plain forms.

Two families, each in both directions:
  attention   causal attention over packed sequences of different lengths, grouped heads:
              gpt2_op_attention_packed_forward / gpt2_op_attention_packed_backward
  logprobs    log-probabilities of given tokens with entropy and the top alternatives:
              gpt2_op_token_logprobs / gpt2_op_token_logprobs_backward
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def attention(name, dir, dtype, n, lo, hi, queries, hq, hkv, hd, mix):
    """n sequences of lo..hi keys (log-uniform, drawn from mix). queries: "all" (a prompt or a training
    document: as many queries as keys), "tail" (a chunk of a prompt whose start is in the cache), "one"
    (one new token each)."""
    return {"name": name, "op": "attention", "dir": dir, "dtype": dtype, "n": n, "lo": lo, "hi": hi,
            "queries": queries, "hq": hq, "hkv": hkv, "hd": hd, "mix": mix}


def logprobs(name, dir, dtype, rows, vocab, padded, top):
    return {"name": name, "op": "logprobs", "dir": dir, "dtype": dtype, "rows": rows, "vocab": vocab,
            "padded": padded, "top": top}


def listed():
    return [
        # a GPT-2 124M training batch of 32 x 1024 tokens as packed documents
        attention("train documents", "forward", "bf16", 62, 100, 1024, "all", 12, 12, 64, 1),
        # prompts from a few tokens to thousands, four query heads to a key head
        attention("ragged prompts", "forward", "bf16", 16, 5, 4096, "all", 16, 4, 64, 2),
        # one step of a served batch: a new token each over caches of up to 8192 tokens
        attention("new tokens", "forward", "bf16", 64, 256, 8192, "one", 16, 4, 64, 3),
        # one new token for a few short sequences of the 124M model: latency
        attention("new token, short", "forward", "bf16", 4, 17, 700, "one", 12, 12, 64, 4),
        # the fp32 mode (exact parity) on packed documents
        attention("fp32 documents", "forward", "f32", 16, 20, 600, "all", 12, 12, 64, 5),
        # the backward pass of the training batch
        attention("train documents, backward", "backward", "bf16", 62, 100, 1024, "all", 12, 12, 64, 1),
        # the fp32 mode's backward pass: chunks after cached keys, shared key heads
        attention("fp32 chunks, backward", "backward", "f32", 9, 3, 400, "tail", 6, 2, 32, 6),
        # scoring every token of the 32 x 1024 batch
        logprobs("score a batch", "forward", "bf16", 32768, 50257, 50304, 0),
        # scoring with the top 20 alternatives of each position, an odd number of rows
        logprobs("alternatives", "forward", "bf16", 2043, 50257, 50304, 20),
        # the next token of a few sequences from fp32 logits: latency
        logprobs("next tokens", "forward", "f32", 8, 50257, 50304, 5),
        # gradients of log-probability and entropy for a batch of 8 x 1024 (policy gradients)
        logprobs("policy gradient", "backward", "bf16", 8192, 50257, 50304, 0),
        # the tiny fp32 model's rows
        logprobs("policy gradient, tiny", "backward", "f32", 256, 512, 512, 0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.6:
        dtype = "bf16" if rng.random() < 0.75 else "f32"
        dir = "forward" if rng.random() < 0.6 else "backward"
        queries = rng.choice(["all", "tail", "one"]) if dir == "forward" else rng.choice(["all", "all", "tail"])
        hq, hkv = rng.choice([(12, 12), (16, 16), (25, 25), (16, 4), (8, 1), (6, 2), (20, 4), (14, 2)])
        hd = 64 if dtype == "bf16" else rng.choice([16, 32, 64])
        most = 600 if dtype == "f32" else 8192 if queries == "one" else 4096
        hi = _log_int(rng, 2, most)
        c = attention("", dir, dtype, _log_int(rng, 1, 64), _log_int(rng, 1, hi), hi, queries, hq, hkv, hd,
                      rng.randrange(1 << 20))
        # no more than the listed ones cost: the padded score matrices and the products
        cap = 2.0e9 if dtype == "bf16" else 1.0e8
        while c["n"] > 1 and c["n"] * hq * float(hi) * (1 if queries == "one" else hi) > cap:
            c["n"] -= 1
    else:
        dtype = "bf16" if rng.random() < 0.7 else "f32"
        dir = "forward" if rng.random() < 0.6 else "backward"
        vocab = rng.choice([50257, _log_int(rng, 300, 50257), _log_int(rng, 300, 50257)])
        rows = _log_int(rng, 1, 8192 if dtype == "bf16" else 4096)
        c = logprobs("", dir, dtype, rows, vocab, -(-vocab // 64) * 64,
                     rng.choice([0, 1, 5, 20, 32]) if dir == "forward" else 0)
    del c["name"]
    return c


def lengths(case):
    """(queries, keys) of each sequence."""
    r = random.Random(case["mix"])
    keys = [_log_int(r, case["lo"], case["hi"]) for _ in range(case["n"])]
    if case["queries"] == "all":
        return list(keys), keys
    if case["queries"] == "one":
        return [1] * len(keys), keys
    return [r.randint(1, x) for x in keys], keys


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "logprobs":
        n, v = case["rows"], case["vocab"]
        if case["dir"] == "forward":
            return {"bytes": n * v * es + n * 4 * (4 + 2 * case["top"]), "flops": 4.0 * n * v}
        return {"bytes": n * v * es + n * case["padded"] * es + n * 20, "flops": 6.0 * n * v}
    lq, lk = lengths(case)
    # query i of a sequence sees the keys 0 .. i + lk - lq
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
    q, kv = sum(lq) * case["hq"] * case["hd"], sum(lk) * case["hkv"] * case["hd"]
    lse = sum(lq) * case["hq"] * 4
    if case["dir"] == "forward":
        return {"bytes": (2 * q + 2 * kv) * es + lse, "flops": 4.0 * case["hd"] * pairs * case["hq"]}
    return {"bytes": (4 * q + 4 * kv) * es + lse, "flops": 10.0 * case["hd"] * pairs * case["hq"]}


# ---------------------------------------------------------------- what a program has in hand

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "logprobs":
        n, v, vp = case["rows"], case["vocab"], case["padded"]
        s = {"case": case}
        z = rand(n, vp)
        z.mul_(2.0).add_(rand(vp) * 1.5)  # frequent and rare tokens, and what a row knows
        s["logits"] = z.to(dt)
        del z
        s["targets"] = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
        s["logp"], s["lse"], s["entropy"] = (torch.zeros(n, device="cuda") for _ in range(3))
        if case["dir"] == "forward":
            s["top_logp"] = torch.zeros(n, case["top"], device="cuda") if case["top"] else None
            s["top_ids"] = torch.zeros(n, case["top"], dtype=torch.int32, device="cuda") if case["top"] else None
        else:
            s["lse"], s["entropy"] = _plain_rows(s["logits"][:, :v].float())[:2]
            s["dlogp"], s["dentropy"] = rand(n) / n, rand(n) * (0.01 / n)
            s["dlogits"] = torch.zeros(n, vp, dtype=dt, device="cuda")
        return s
    lq, lk = lengths(case)
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    tq, tk = sum(lq), sum(lk)

    def offsets(x):
        at = [0]
        for y in x:
            at.append(at[-1] + y)
        return torch.tensor(at, dtype=torch.int32, device="cuda")

    s = {"case": case, "cu_q": offsets(lq), "cu_k": offsets(lk), "max_q": max(lq), "max_k": max(lk)}

    def heads(x, first, count):  # `count` heads of x's rows from head `first` on
        return x[:, first * hd:(first + count) * hd].unflatten(1, (count, hd))

    if case["queries"] == "all":  # the fused projection's output, as the model has it
        x = rand(tq, (hq + 2 * hkv) * hd).to(dt)
        s["q"], s["k"], s["v"] = heads(x, 0, hq), heads(x, hq, hkv), heads(x, hq + hkv, hkv)
    else:
        x = rand(tk, 2 * hkv * hd).to(dt)
        s["q"] = rand(tq, hq, hd).to(dt)
        s["k"], s["v"] = heads(x, 0, hkv), heads(x, hkv, hkv)
    s["o"] = torch.zeros(tq, hq, hd, dtype=dt, device="cuda")
    s["lse"] = torch.zeros(hq, tq, device="cuda")
    if case["dir"] == "backward":
        s["dout"] = rand(tq, hq, hd).to(dt)
        s["o"], s["lse"] = _plain_attention(s)  # the forward's outputs
        if case["queries"] == "all":
            d = torch.zeros(tq, (hq + 2 * hkv) * hd, dtype=dt, device="cuda")
            s["dq"], s["dk"], s["dv"] = heads(d, 0, hq), heads(d, hq, hkv), heads(d, hq + hkv, hkv)
        else:
            s["dq"] = torch.zeros(tq, hq, hd, dtype=dt, device="cuda")
            s["dk"], s["dv"] = (torch.zeros(tk, hkv, hd, dtype=dt, device="cuda") for _ in range(2))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        from step_gpt_train_gb300 import gpt2 as g
        if case["op"] == "attention":
            if case["dir"] == "forward":
                g.gpt2_op_attention_packed_forward(s["o"], s["lse"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                                   s["max_q"], s["max_k"])
                return {"o": s["o"], "lse": s["lse"]}
            g.gpt2_op_attention_packed_backward(s["dq"], s["dk"], s["dv"], s["dout"], s["q"], s["k"], s["v"], s["o"],
                                                s["lse"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"])
            return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
        if case["dir"] == "forward":
            g.gpt2_op_token_logprobs(s["logp"], s["lse"], s["entropy"], s["logits"], s["targets"], case["vocab"],
                                     top_logp=s["top_logp"], top_ids=s["top_ids"])
            return {"logp": s["logp"], "lse": s["lse"], "entropy": s["entropy"], "top_logp": s["top_logp"],
                    "top_ids": s["top_ids"]}
        g.gpt2_op_token_logprobs_backward(s["dlogits"], s["logits"], s["targets"], s["lse"], s["entropy"],
                                          case["vocab"], dlogp=s["dlogp"], dentropy=s["dentropy"])
        return {"dlogits": s["dlogits"]}
    if case["op"] == "attention":
        if case["dir"] == "forward":
            o, lse = _plain_attention(s)
            return {"o": o, "lse": lse}
        dq, dk, dv = _plain_attention_backward(s)
        return {"dq": dq, "dk": dk, "dv": dv}
    return _plain_logprobs(s) if case["dir"] == "forward" else _plain_logprobs_backward(s)


def _padded(s):
    """The sequences side by side: row numbers, which of them are real, and which key a query sees."""
    dev = s["cu_q"].device
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    i, j = torch.arange(s["max_q"], device=dev), torch.arange(s["max_k"], device=dev)
    real_q, real_k = i[None] < lq[:, None], j[None] < lk[:, None]
    at_q = torch.where(real_q, cq[:-1, None] + i, 0)
    at_k = torch.where(real_k, ck[:-1, None] + j, 0)
    sees = real_q[:, :, None] & (j[None, None] <= i[None, :, None] + (lk - lq)[:, None, None])
    return at_q, real_q, at_k, real_k, sees[:, None, None]


def _scores(s, at_q, at_k, sees):
    hq, hkv, hd = s["case"]["hq"], s["case"]["hkv"], s["case"]["hd"]
    q = s["q"][at_q].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4)  # [n, hkv, group, Lq, hd]
    k = s["k"][at_k].float().permute(0, 2, 1, 3)[:, :, None]                        # [n, hkv, 1, Lk, hd]
    x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
    return q, k, x.masked_fill_(~sees, -math.inf)


def _plain_attention(s):
    at_q, real_q, at_k, real_k, sees = _padded(s)
    _, _, x = _scores(s, at_q, at_k, sees)
    m = x.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
    p = torch.exp(x.sub_(m))
    total = p.sum(-1, keepdim=True)
    v = s["v"][at_k].float().permute(0, 2, 1, 3)[:, :, None]
    y = (p @ v) / total.clamp_min(1e-30)
    o, lse = torch.zeros_like(s["o"]), torch.zeros_like(s["lse"])
    hq = s["case"]["hq"]
    at = at_q[real_q]
    o[at] = y.permute(0, 3, 1, 2, 4).flatten(2, 3)[real_q].to(o.dtype)
    lse[:, at] = (m + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(*at_q.shape, hq)[real_q].T
    return o, lse


def _plain_attention_backward(s):
    case = s["case"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    at_q, real_q, at_k, real_k, sees = _padded(s)
    q, k, x = _scores(s, at_q, at_k, sees)
    split = lambda t: t.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4)  # noqa: E731
    lse = s["lse"].T[at_q].unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1)[..., None]
    p = torch.exp(x - lse.nan_to_num(neginf=0.0))
    dy = split(torch.where(real_q[:, :, None, None], s["dout"][at_q].float(), 0.0))
    d = (dy * split(s["o"][at_q].float())).sum(-1, keepdim=True)
    v = s["v"][at_k].float().permute(0, 2, 1, 3)[:, :, None]
    dv = (p.transpose(-1, -2) @ dy).sum(2)
    ds = p * (dy @ v.transpose(-1, -2) - d) * (1.0 / math.sqrt(hd))
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    dt = s["q"].dtype
    out_q = torch.zeros(s["q"].shape, dtype=dt, device=q.device)
    out_k, out_v = (torch.zeros(s["k"].shape, dtype=dt, device=q.device) for _ in range(2))
    out_q[at_q[real_q]] = dq.permute(0, 3, 1, 2, 4).flatten(2, 3)[real_q].to(dt)
    out_k[at_k[real_k]] = dk.permute(0, 2, 1, 3)[real_k].to(dt)
    out_v[at_k[real_k]] = dv.permute(0, 2, 1, 3)[real_k].to(dt)
    return out_q, out_k, out_v


def _plain_rows(z):
    """lse, entropy and log-probabilities of fp32 rows."""
    m = z.amax(-1, keepdim=True)
    lse = m + torch.exp(z - m).sum(-1, keepdim=True).log()
    lp = z - lse
    return lse.squeeze(-1), -(torch.exp(lp) * lp).sum(-1), lp


def _plain_logprobs(s):
    case = s["case"]
    z = s["logits"][:, :case["vocab"]].float()
    lse, entropy, lp = _plain_rows(z)
    out = {"logp": lp.gather(1, s["targets"].long()[:, None]).squeeze(1), "lse": lse, "entropy": entropy,
           "top_logp": None, "top_ids": None}
    if case["top"]:
        # the value's order in the high half, the lowest index first in the low half
        b = (z + 0.0).view(torch.int32)
        order = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * (1 << 32)
        order += (1 << 31) - torch.arange(z.shape[1], device=z.device)
        ids = order.topk(case["top"], dim=1).indices
        out["top_logp"], out["top_ids"] = lp.gather(1, ids), ids.int()
    return out


def _plain_logprobs_backward(s):
    case = s["case"]
    v = case["vocab"]
    lp = s["logits"][:, :v].float() - s["lse"][:, None]
    p = torch.exp(lp)
    g = -p * (s["dlogp"][:, None] + s["dentropy"][:, None] * (lp + s["entropy"][:, None]))
    g.scatter_add_(1, s["targets"].long()[:, None], s["dlogp"][:, None])
    out = torch.zeros_like(s["logits"])
    out[:, :v] = g.to(out.dtype)
    return {"dlogits": out}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attention(s) if case["op"] == "attention" else _exact_logprobs(s)


def _exact_attention(s):
    case = s["case"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    back = case["dir"] == "backward"
    o, lse = torch.zeros_like(q), torch.zeros(hq, q.shape[0], dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = b = 0
    for nq, nk in zip(*lengths(case)):
        rows, keys = torch.arange(nq, device=q.device), torch.arange(nk, device=q.device)
        hidden = keys[None, :] - rows[:, None] > nk - nq
        for h in range(hkv):
            kh, vh = k[b:b + nk, h], v[b:b + nk, h]
            for u in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = torch.einsum("id,jd->ij", q[a:a + nq, u], kh) / hd ** 0.5
                x[hidden] = -math.inf
                lse[u, a:a + nq] = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
                o[a:a + nq, u] = w @ vh
                if back:
                    dy = s["dout"][a:a + nq, u].double()
                    dv[b:b + nk, h] += w.T @ dy
                    dw = dy @ vh.T
                    dx = w * (dw - (w * dw).sum(1, keepdim=True)) / hd ** 0.5
                    dq[a:a + nq, u] = dx @ kh
                    dk[b:b + nk, h] += dx.T @ q[a:a + nq, u]
        a, b = a + nq, b + nk
    return {"dq": dq, "dk": dk, "dv": dv} if back else {"o": o, "lse": lse}


def _exact_logprobs(s):
    case = s["case"]
    n, v = case["rows"], case["vocab"]
    lp = torch.log_softmax(s["logits"][:, :v].double(), 1)
    at = s["targets"].long()
    rows = torch.arange(n, device=lp.device)
    if case["dir"] == "forward":
        top = torch.sort(lp, 1, descending=True).values[:, :case["top"]] if case["top"] else None
        return {"logp": lp[rows, at], "lse": torch.logsumexp(s["logits"][:, :v].double(), 1),
                "entropy": -torch.special.xlogy(lp.exp(), lp.exp()).sum(1), "top_logp": top, "top_ids": None}
    p = lp.exp()
    h = -(p * lp).sum(1)
    out = torch.zeros(n, case["padded"], dtype=torch.float64, device=lp.device)
    out[rows, at] = s["dlogp"].double()
    out[:, :v] -= s["dlogp"].double()[:, None] * p
    out[:, :v] -= s["dentropy"].double()[:, None] * p * (lp + h[:, None])
    return {"dlogits": out}
