"""Cases of what a training step over packed documents needs beside attention, with their plain forms.

Three families:
  rotary      norms of queries and keys for each head with the position rotation, in both directions:
              gpt2_op_qk_norm_rotary_forward / gpt2_op_qk_norm_rotary_backward
  loss        softmax cross entropy from hidden states and the head's weight without keeping the logits,
              in both directions: gpt2_op_linear_classifier_forward / gpt2_op_linear_classifier_backward
  adamw       AdamW over many tensors at once, with moments in 32 or in 8 bits:
              gpt2_op_adamw_many (and gpt2_op_adamw_many_states, which reads 8-bit moments back)
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def rotary(name, dir, dtype, rows, hq, hk, hd, rot, layout, norm, scaling, reach, fused):
    """rows tokens of hq query and hk key heads; the first rot values of a head are rotated, as pairs of
    values half of rot apart ("half") or next to each other ("interleaved"). scaling: how the frequencies
    are stretched for long contexts. reach: the furthest position. fused: queries and keys are column blocks
    of the qkv projection's output."""
    return {"name": name, "op": "rotary", "dir": dir, "dtype": dtype, "rows": rows, "hq": hq, "hk": hk, "hd": hd,
            "rot": rot, "layout": layout, "norm": norm, "scaling": scaling, "reach": reach, "fused": fused}


def loss(name, dir, dtype, rows, width, vocab, padded):
    return {"name": name, "op": "loss", "dir": dir, "dtype": dtype, "rows": rows, "width": width, "vocab": vocab,
            "padded": padded}


def adamw(name, bits, grads, tensors, clip):
    """tensors: "model L C V T" (the tensors of a GPT-2 of L layers) or "mix K LO HI S" (K tensors of LO..HI
    values, log-uniform, drawn from S)."""
    return {"name": name, "op": "adamw", "bits": bits, "grads": grads, "tensors": tensors, "clip": clip}


def listed():
    return [
        # the training batch of 32 x 1024 tokens, twelve heads in the fused qkv buffer
        rotary("rotate a batch", "forward", "bf16", 32768, 12, 12, 64, 64, "half", True, "none", 1024, True),
        # its backward pass, with the gradients of the norms' weights
        rotary("rotate a batch, backward", "backward", "bf16", 32768, 12, 12, 64, 64, "half", True, "none", 1024, True),
        # one new token for each of 64 served sequences, far positions, half of the head rotated: latency
        rotary("rotate new tokens", "forward", "bf16", 64, 16, 4, 64, 32, "interleaved", False, "parts", 131072, False),
        # the fp32 mode on shared key heads, an odd number of rows
        rotary("rotate fp32, backward", "backward", "f32", 4001, 6, 2, 32, 32, "interleaved", True, "linear", 16384,
               False),
        # the loss of the 32 x 1024 batch of the 124M model
        loss("loss of a batch", "forward", "bf16", 32768, 768, 50257, 50304),
        # the gradients of the 8 x 1024 batch
        loss("loss, backward", "backward", "bf16", 8192, 768, 50257, 50304),
        # scoring the last tokens of a few prompts: latency, the weight is read once
        loss("loss of few rows", "forward", "bf16", 61, 768, 50257, 50304),
        # a small fp32 model with an odd vocabulary
        loss("loss fp32, backward", "backward", "f32", 1021, 128, 5003, 5056),
        # the 124M model's tensors with clipping, moments in 32 bits
        adamw("update 124M", 32, "f32", "model 12 768 50304 1024", True),
        # the same with moments in 8 bits
        adamw("update 124M, 8 bits", 8, "f32", "model 12 768 50304 1024", True),
        # a tiny model's tensors: latency
        adamw("update a tiny model", 32, "f32", "model 2 128 512 128", False),
        # tensors of odd sizes, bf16 gradients, moments in 8 bits
        adamw("update odd tensors, 8 bits", 8, "bf16", "mix 37 1 300000 5", False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotary", "loss", "adamw"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    dir = rng.choice(["forward", "backward"])
    if kind == "rotary":
        hq, hk = rng.choice([(12, 12), (16, 16), (25, 25), (16, 4), (8, 1), (6, 2), (14, 2)])
        hd = 64 if dtype == "bf16" else rng.choice([16, 32, 64])
        rot = rng.choice([hd, hd, hd // 2, hd // 4 // 8 * 8 or 8])
        c = rotary("", dir, dtype, _log_int(rng, 1, 32768 * 24 // (hq + hk) // (1 if dtype == "bf16" else 2)), hq, hk, hd,
                   rot, rng.choice(["half", "interleaved"]), rng.random() < 0.7,
                   rng.choice(["none", "linear", "base", "parts"]), _log_int(rng, 128, 262144), rng.random() < 0.5)
    elif kind == "loss":
        width = 8 * _log_int(rng, 8, 200 if dtype == "bf16" else 48)
        vocab = rng.choice([50257, _log_int(rng, 300, 50257), _log_int(rng, 300, 50257)])
        # no more than the listed ones cost
        most = (1.2e12 if dir == "forward" else 3.0e11) if dtype == "bf16" else 6.0e9
        c = loss("", dir, dtype, _log_int(rng, 1, max(1, min(32768, int(most / width / vocab)))), width, vocab,
                 -(-vocab // 64) * 64)
    else:
        c = adamw("", rng.choice([8, 8, 32]), "bf16" if rng.random() < 0.4 else "f32",
                  "mix %d %d %d %d" % (_log_int(rng, 1, 200), rng.choice([1, 64, 1000]), _log_int(rng, 2000, 600000),
                                       rng.randrange(1 << 20)), rng.random() < 0.5)
    del c["name"]
    return c


def sizes(case):
    """(values, whether weight decay applies) of each tensor of an adamw case."""
    kind, *a = case["tensors"].split()
    a = [int(x) for x in a]
    if kind == "model":
        layers, c, vocab, ctx = a
        one = [(c, False), (c, False), (3 * c * c, True), (3 * c, False), (c * c, True), (c, False), (c, False),
               (c, False), (4 * c * c, True), (4 * c, False), (4 * c * c, True), (c, False)]
        return [(vocab * c, True), (ctx * c, True)] + layers * one + [(c, False), (c, False)]
    r = random.Random(a[3])
    return [(_log_int(r, a[1], a[2]), r.random() < 0.7) for _ in range(a[0])]


def work(case):
    if case["op"] == "rotary":
        n = case["rows"] * (case["hq"] + case["hk"]) * case["hd"] * SIZE[case["dtype"]]
        back = case["dir"] == "backward"
        # the gradients' way back reads x too where it has a norm
        return {"bytes": n * (2 + (back and case["norm"])) + 4 * case["rows"],
                "flops": (20.0 if back else 10.0) * n / SIZE[case["dtype"]]}
    if case["op"] == "loss":
        es, n, c, v = SIZE[case["dtype"]], case["rows"], case["width"], case["vocab"]
        if case["dir"] == "forward":
            return {"bytes": (n + v) * c * es + 12 * n, "flops": 2.0 * n * c * v}
        # the logits once more, then both gradients
        return {"bytes": 2 * (n + v) * c * es + 12 * n, "flops": 6.0 * n * c * v}
    n = sum(x for x, _ in sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 4 / 128
    # clipping reads the gradients before the first of them is used; 8-bit moments are read back as bf16
    g = SIZE[case["grads"]] * (2 if case["clip"] else 1)
    return {"bytes": n * (8 + 2 + g + state + (6 if case["bits"] == 8 else 0)), "flops": 15.0 * n}


# ---------------------------------------------------------------- what a program has in hand

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    return {"rotary": _prepare_rotary, "loss": _prepare_loss, "adamw": _prepare_adamw}[case["op"]](case, seed, gen, rand)


def _turns(rot, scaling):
    """Turns of each pair from one position to the next, in units of 2^-64."""
    base, factor, context, fast, slow = 10000.0, 8.0, 8192, 32.0, 1.0
    if scaling == "base":
        base *= factor ** (rot / max(rot - 2, 1))
    out = []
    for j in range(rot // 2):
        f = base ** (-2.0 * j / rot) / (2 * math.pi)
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            keep = min(1.0, max(0.0, (f * context - slow) / (fast - slow)))
            f *= keep + (1 - keep) / factor
        out.append(round(f * 2.0 ** 64))
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def _prepare_rotary(case, seed, gen, rand):
    n, hq, hk, hd, dt = case["rows"], case["hq"], case["hk"], case["hd"], DT[case["dtype"]]
    s = {"case": case, "turns": _turns(case["rot"], case["scaling"]), "eps": 1e-6 if case["norm"] else None,
         "amplitude": 0.1 * math.log(8.0) + 1 if case["scaling"] == "parts" else 1.0}
    # packed documents: each counts its positions from a start of its own
    start = torch.randint(0, case["reach"], (n,), generator=gen, device="cuda")
    s["pos"] = ((torch.arange(n, device="cuda") % 700 + start[torch.arange(n, device="cuda") // 700]) % case["reach"]).int()

    def pair(std):
        if not case["fused"]:
            return (rand(n, hq, hd) * std).to(dt), (rand(n, hk, hd) * std).to(dt)
        x = (rand(n, (hq + 2 * hk) * hd) * std).to(dt)
        return x[:, :hq * hd].unflatten(1, (hq, hd)), x[:, hq * hd:(hq + hk) * hd].unflatten(1, (hk, hd))

    s["q"], s["k"] = pair(1.5)
    s["q_gamma"], s["k_gamma"] = ((1 + 0.1 * rand(hd)).to(dt) if case["norm"] else None for _ in range(2))
    if case["dir"] == "forward":
        s["qo"], s["ko"] = torch.zeros(n, hq, hd, dtype=dt, device="cuda"), torch.zeros(n, hk, hd, dtype=dt, device="cuda")
        return s
    s["dqo"], s["dko"] = rand(n, hq, hd).to(dt), rand(n, hk, hd).to(dt)
    s["dq"], s["dk"] = pair(0.0)
    s["dq_gamma"], s["dk_gamma"] = (torch.zeros(hd, device="cuda") if case["norm"] else None for _ in range(2))
    return s


def _prepare_loss(case, seed, gen, rand):
    n, c, v, vp, dt = case["rows"], case["width"], case["vocab"], case["padded"], DT[case["dtype"]]
    s = {"case": case, "x": rand(n, c).to(dt)}
    w = rand(vp, c) * (2.5 / math.sqrt(c))
    w[v:] = 0
    s["w"] = w.to(dt)
    s["targets"] = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    s["losses"], s["lse"] = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    if case["dir"] == "backward":
        s["lse"] = _plain_loss(s)["lse"]
        # the mean over the tokens that count; a fifth of them is a prompt or padding
        s["dloss"] = (torch.rand(n, generator=gen, device="cuda") < 0.8).float() / n
        s["dx"], s["dw"] = torch.zeros_like(s["x"]), torch.zeros_like(s["w"])
    return s


BLOCK = 128  # values of an 8-bit moment that share a scale


def _prepare_adamw(case, seed, gen, rand):
    each = sizes(case)
    at = [0]  # each tensor starts on a block's border of a common buffer
    for n, _ in each:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    blocks = torch.tensor([-(-n // BLOCK) for n, _ in each], device="cuda")
    per_block = lambda x: torch.repeat_interleave(x, blocks)[:, None]  # noqa: E731
    s = {"case": case, "lr": 6e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "t": 100 + seed % 1000, "grad_scale": 0.5,
         "max_grad_norm": 1.0 if case["clip"] else 0.0, "seed": seed}
    s["decay"] = [0.1 if d else 0.0 for _, d in each]
    s["decay_of"] = per_block(torch.tensor(s["decay"], device="cuda"))
    s["tensor_of"] = per_block(torch.arange(len(each), device="cuda"))
    first = torch.tensor(at[:-1], device="cuda") // BLOCK
    s["block_of"] = torch.arange(at[-1] // BLOCK, device="cuda")[:, None] - per_block(first)
    left = per_block(torch.tensor([n for n, _ in each], device="cuda")) - s["block_of"] * BLOCK
    real = torch.arange(BLOCK, device="cuda")[None] < left
    size = torch.exp(-8 + 2.5 * rand(len(each)).clamp(-2, 2))  # gradients of different tensors differ in size
    size = per_block(size) * real
    nb = at[-1] // BLOCK
    s["master"] = 0.02 * rand(nb, BLOCK) * real
    s["param"] = s["master"].to(torch.bfloat16)
    s["grad"] = (2 * size * rand(nb, BLOCK)).to(DT[case["grads"]])
    m, v = 0.3 * size * rand(nb, BLOCK), size * size * (0.3 + torch.rand(nb, BLOCK, generator=gen, device="cuda"))
    if case["bits"] == 8:
        half = torch.tensor(0.5, device="cuda")
        (s["m"], s["m_scale"]), (s["v"], s["v_scale"]) = _encode(m, half, M8), _encode(v, half, V8)
        s["m_values"], s["v_values"] = (torch.zeros(nb, BLOCK, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        s["m"], s["v"] = m, v
    s["norm"] = torch.zeros(1, device="cuda")

    def apart(name, per=1):
        flat = s[name].view(-1)
        return [flat[a // per:a // per + -(-n // per)] for a, (n, _) in zip(at, each)]

    s["tensors"] = {"masters": apart("master"), "grads": apart("grad"), "ms": apart("m"), "vs": apart("v"),
                    "params": apart("param"), "weight_decay": s["decay"]}
    if case["bits"] == 8:
        s["tensors"] |= {"m_scales": apart("m_scale", BLOCK), "v_scales": apart("v_scale", BLOCK),
                         "m_values": apart("m_values"), "v_values": apart("v_values")}
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        from step_gpt_train_gb300 import gpt2 as g
        if case["op"] == "rotary":
            kw = {"q_gamma": s["q_gamma"], "k_gamma": s["k_gamma"], "eps": s["eps"],
                  "interleaved": case["layout"] == "interleaved", "amplitude": s["amplitude"]}
            if case["dir"] == "forward":
                g.gpt2_op_qk_norm_rotary_forward(s["qo"], s["ko"], s["q"], s["k"], s["pos"], s["turns"], **kw)
                return {"q": s["qo"], "k": s["ko"]}
            g.gpt2_op_qk_norm_rotary_backward(s["dq"], s["dk"], s["dqo"], s["dko"], s["q"], s["k"], s["pos"], s["turns"],
                                              dq_gamma=s["dq_gamma"], dk_gamma=s["dk_gamma"], **kw)
            return {"dq": s["dq"], "dk": s["dk"], "dq_gamma": s["dq_gamma"], "dk_gamma": s["dk_gamma"]}
        if case["op"] == "loss":
            if case["dir"] == "forward":
                g.gpt2_op_linear_classifier_forward(s["losses"], s["lse"], s["x"], s["w"], s["targets"], case["vocab"])
                return {"losses": s["losses"], "lse": s["lse"]}
            g.gpt2_op_linear_classifier_backward(s["dx"], s["dw"], s["x"], s["w"], s["targets"], s["lse"], case["vocab"],
                                                 dloss=s["dloss"])
            return {"dx": s["dx"], "dw": s["dw"]}
        if "handle" not in s:  # the program's list of its tensors, made once
            s["handle"] = g.gpt2_adamw_tensors(**s["tensors"])
        g.gpt2_op_adamw_many(s["handle"], s["lr"], s["beta1"], s["beta2"], s["eps"], s["t"], grad_scale=s["grad_scale"],
                             max_grad_norm=s["max_grad_norm"], grad_norm=s["norm"] if case["clip"] else None,
                             seed=s["seed"])
        if case["bits"] == 8:
            g.gpt2_op_adamw_many_states(s["handle"])
        return _updated(s)
    if case["op"] == "rotary":
        return _plain_rotary(s) if case["dir"] == "forward" else _plain_rotary_backward(s)
    if case["op"] == "loss":
        return _plain_loss(s) if case["dir"] == "forward" else _plain_loss_backward(s)
    return _plain_adamw(s)


def _updated(s):
    m, v = ("m_values", "v_values") if s["case"]["bits"] == 8 else ("m", "v")
    return {"master": s["master"], "param": s["param"], "m": s[m], "v": s[v],
            "norm": s["norm"] if s["case"]["clip"] else None}


def _angles(s):
    """cos and sin of each row's rotation, [rows, 1, rot / 2], times the amplitude; the angles in 64 bits."""
    turned = s["pos"].double()[:, None] * (s["turns"].double() * 2.0 ** -64)
    a = (turned - turned.round()) * (2 * math.pi)
    return (a.cos() * s["amplitude"]).float()[:, None], (a.sin() * s["amplitude"]).float()[:, None]


def _pairs(s, x):
    """The first and second values of the pairs, and the rest of the head."""
    r = s["case"]["rot"]
    if s["case"]["layout"] == "half":
        return x[..., :r // 2], x[..., r // 2:r], x[..., r:]
    return x[..., :r:2], x[..., 1:r:2], x[..., r:]


def _joined(s, a, b, rest):
    if s["case"]["layout"] == "half":
        return torch.cat((a, b, rest), -1)
    return torch.cat((torch.stack((a, b), -1).flatten(-2), rest), -1)


def _plain_rotary(s):
    cos, sin = _angles(s)

    def one(x, gamma):
        x = x.float()
        if s["eps"] is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * gamma.float()
        a, b, rest = _pairs(s, x)
        return _joined(s, a * cos - b * sin, a * sin + b * cos, rest)

    dt = s["q"].dtype
    return {"q": one(s["q"], s["q_gamma"]).to(dt), "k": one(s["k"], s["k_gamma"]).to(dt)}


def _plain_rotary_backward(s):
    cos, sin = _angles(s)

    def one(dy, x, gamma):
        a, b, rest = _pairs(s, dy.float())
        dn = _joined(s, a * cos + b * sin, b * cos - a * sin, rest)
        if s["eps"] is None:
            return dn.to(dy.dtype), None
        x = x.float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        xhat = x * rstd
        d = dn * gamma.float()
        dx = rstd * (d - xhat * (d * xhat).mean(-1, keepdim=True))
        return dx.to(dy.dtype), (dn * xhat).sum((0, 1))

    dq, dqg = one(s["dqo"], s["q"], s["q_gamma"])
    dk, dkg = one(s["dko"], s["k"], s["k_gamma"])
    return {"dq": dq, "dk": dk, "dq_gamma": dqg, "dk_gamma": dkg}


def _logits(s):
    return s["x"].float() @ s["w"][:s["case"]["vocab"]].float().T


def _plain_loss(s):
    z = _logits(s)
    m = z.amax(-1)
    at = z.gather(1, s["targets"].long()[:, None]).squeeze(1)
    lse = z.sub_(m[:, None]).exp_().sum(-1).log() + m
    return {"losses": lse - at, "lse": lse}


def _plain_loss_backward(s):
    v = s["case"]["vocab"]
    dz = _logits(s).sub_(s["lse"][:, None]).exp_().mul_(s["dloss"][:, None])
    dz.scatter_add_(1, s["targets"].long()[:, None], -s["dloss"][:, None])
    dw = torch.zeros_like(s["w"])
    dw[:v] = (dz.T @ s["x"].float()).to(dw.dtype)
    return {"dx": (dz @ s["w"][:v].float()).to(s["x"].dtype), "dw": dw}


# 8-bit floating point codes of three mantissa bits: (exponent bias, sign bit, exponent of a block's largest value)
M8 = (7, 0x80, 7)     # e4m3: sign, 4 exponent bits
V8 = (15, 0, 14)      # e5m3: no sign, 5 exponent bits; a value above 0 keeps at least the lowest code


def _power(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, u, kind):
    """Codes of blocks [nb, BLOCK] and each block's scale (a power of two, as its exponent + 127): a value goes up
    with u in [0, 1) above what is left of it on the way down."""
    bias, sign, top = kind
    size = x.abs()
    largest = torch.frexp(size.amax(-1, keepdim=True)).exponent - 1
    scale = (largest - top + 127).clamp(1, 254)
    y = size * _power(127 - scale)
    e = torch.where(y > 0, torch.frexp(y).exponent - 1, 1 - bias).clamp_min(1 - bias)
    k = torch.floor(y * _power(3 - e) + u)  # eighths of 2^e: 0 .. 16
    code = ((e + bias - 1) * 8 + k).int()   # the same for what is below the lowest whole exponent
    if sign:
        code = torch.where(x < 0, code | sign, code)
    else:
        code = torch.where((x > 0) & (code == 0), 1, code)
    return code.to(torch.uint8), scale.to(torch.uint8)


def _decode(code, scale, kind):
    bias, sign, _ = kind
    c = code.int()
    k = c & 127 if sign else c
    e = (k >> 3).clamp_min(1)
    y = (torch.where(k >= 8, 8, 0) + (k & 7)).float() * _power(e - bias - 3) * _power(scale.int().clamp_min(1) - 127)
    return torch.where((c & sign) != 0, -y, y) if sign else y


GOLDEN, MIX1, MIX2 = (x - (1 << 64) for x in (0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB))


def _mix(z):
    """The finaliser of splitmix64 on int64 tensors."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * MIX1
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * MIX2
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _uniforms(s):
    """For each value of the blocks: 16 bits for the first moment's rounding and 16 for the second's, as numbers in
    [0, 1); two neighbours share one draw."""
    key = _mix(torch.tensor(s["seed"], device="cuda") + s["t"] * torch.tensor(GOLDEN, device="cuda"))
    pair = s["block_of"] * (BLOCK // 2) + torch.arange(BLOCK // 2, device="cuda")
    r = _mix(key + ((s["tensor_of"] << 40) + pair) * GOLDEN)
    part = lambda n: ((r >> n) & 0xFFFF).float() * 2.0 ** -16  # noqa: E731
    return torch.stack((part(0), part(32)), -1).flatten(1), torch.stack((part(16), part(48)), -1).flatten(1)


def _f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def _plain_adamw(s):
    case = s["case"]
    b1, b2, eps, lr = (_f32(s[k]) for k in ("beta1", "beta2", "eps", "lr"))
    g = s["grad"].float()
    scale = s["grad_scale"]
    if case["clip"]:
        s["norm"][0] = g.double().square().sum().sqrt()
        scale = scale * (s["max_grad_norm"] / (s["norm"] * scale + 1e-6)).clamp_max(1.0)
    g = g * scale
    m, v = (s["m"], s["v"]) if case["bits"] == 32 else (_decode(s["m"], s["m_scale"], M8),
                                                         _decode(s["v"], s["v_scale"], V8))
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    step = m / (1 - b1 ** s["t"]) / (torch.sqrt(v / (1 - b2 ** s["t"])) + eps)
    s["master"] -= lr * (step + s["decay_of"] * s["master"])
    s["param"].copy_(s["master"])
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _updated(s)
    um, uv = _uniforms(s)
    for x, u, name, kind in ((m, um, "m", M8), (v, uv, "v", V8)):
        code, power = _encode(x, u, kind)
        s[name].copy_(code)
        s[name + "_scale"].copy_(power)
        s[name + "_values"].copy_(_decode(s[name], s[name + "_scale"], kind))
    return _updated(s)


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "loss": _exact_loss, "adamw": _exact_adamw}[case["op"]](s)


def _exact_rotary(s):
    case = s["case"]
    rot, hd = case["rot"], case["hd"]
    back = case["dir"] == "backward"
    out = {}
    lead = range(rot // 2) if case["layout"] == "half" else range(0, rot, 2)
    i = torch.tensor(list(lead), device="cuda")
    j = i + (rot // 2 if case["layout"] == "half" else 1)
    w = torch.polar(torch.full((case["rows"], 1, rot // 2), float(s["amplitude"]), dtype=torch.float64, device="cuda"),
                    2 * math.pi * torch.fmod(s["pos"].double()[:, None, None] * (s["turns"].double() / 2.0 ** 64), 1.0))
    for name in ("q", "k"):
        x = s[name].double()
        n = x
        if case["norm"]:
            gamma = s[name + "_gamma"].double()
            r = 1 / torch.sqrt((x ** 2).sum(2, keepdim=True) / hd + s["eps"])
            n = x * r * gamma
        if not back:
            y = n.clone()
            turned = torch.complex(n[..., i], n[..., j]) * w
            y[..., i], y[..., j] = turned.real, turned.imag
            out[name] = y
            continue
        dy = s["d" + name + "o"].double()
        dn = dy.clone()
        turned = torch.complex(dy[..., i], dy[..., j]) * w.conj()
        dn[..., i], dn[..., j] = turned.real, turned.imag
        out["d" + name + "_gamma"] = None
        if case["norm"]:
            out["d" + name + "_gamma"] = torch.einsum("nhd,nhd->d", dn, x * r)
            inner = torch.einsum("nhd,nhd->nh", dn * gamma, x)[..., None]
            dn = dn * gamma * r - x * r ** 3 * inner / hd
        out["d" + name] = dn
    return out


def _exact_loss(s):
    case = s["case"]
    v = case["vocab"]
    w = s["w"][:v].double()
    losses, lses, dx, dw = [], [], [], torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    for a in range(0, case["rows"], 4096):
        x, t = s["x"][a:a + 4096].double(), s["targets"][a:a + 4096].long()
        lp = torch.log_softmax(torch.einsum("nc,vc->nv", x, w), 1)
        row = torch.arange(len(t), device="cuda")
        if case["dir"] == "forward":
            losses.append(-lp[row, t])
            lses.append(torch.einsum("nc,nc->n", x, w[t]) - lp[row, t])
            continue
        d = s["dloss"][a:a + 4096].double()
        dz = lp.exp() * d[:, None]
        dz[row, t] -= d
        dx.append(torch.einsum("nv,vc->nc", dz, w))
        dw[:v] += torch.einsum("nv,nc->vc", dz, x)
    if case["dir"] == "forward":
        return {"losses": torch.cat(losses), "lse": torch.cat(lses)}
    return {"dx": torch.cat(dx), "dw": dw}


def _exact_adamw(s):
    case = s["case"]
    b1, b2, eps, lr = (torch.tensor(s[k], dtype=torch.float32).double().item() for k in ("beta1", "beta2", "eps", "lr"))
    g = s["grad"].double()
    norm = torch.linalg.vector_norm(g)
    factor = s["grad_scale"]
    if case["clip"]:
        factor = factor * min(1.0, s["max_grad_norm"] / (norm.item() * factor + 1e-6))
    g *= factor

    def value(code, scale, bias, signed):
        c = code.long()
        k = c % 128 if signed else c
        e, f = k // 8, (k % 8).double() / 8
        y = torch.where(e > 0, (1 + f) * torch.exp2((e - bias).double()), f * 2.0 ** (1 - bias))
        return y * torch.exp2(scale.double() - 127) * (torch.where(c >= 128, -1.0, 1.0) if signed else 1.0)

    def rounded(x, u, bias, largest, floor):
        # the block's largest value into [2^largest, 2^(largest + 1)), then to multiples of an eighth of the binade
        lg = torch.floor(torch.log2(x.abs().amax(1, keepdim=True).clamp_min(1e-300)))
        unit = torch.exp2((lg - largest).clamp(-126, 127))
        y = x.abs() / unit
        step = torch.exp2(torch.floor(torch.log2(y.clamp_min(1e-300))).clamp_min(1 - bias) - 3)
        k = torch.floor(y / step + u) * step
        if floor:
            k = torch.where((x > 0) & (k == 0), 2.0 ** (1 - bias - 3), k)
        return torch.sign(x) * k * unit

    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m, v = value(s["m"], s["m_scale"], 7, True), value(s["v"], s["v_scale"], 15, False)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    th = s["master"].double()
    th = th - lr * (m / (1 - b1 ** s["t"]) / ((v / (1 - b2 ** s["t"])).sqrt() + eps)
                    + s["decay_of"].double() * th)
    if case["bits"] == 8:
        um, uv = _uniforms(s)
        m, v = rounded(m, um.double(), 7, 7, False), rounded(v, uv.double(), 15, 14, True)
    return {"master": th, "param": th, "m": m, "v": v, "norm": norm.reshape(1) if case["clip"] else None}
