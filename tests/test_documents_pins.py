"""Pins of the oracle of head norms with rotary positions, the cross entropy of hidden states and AdamW over many
tensors (CPU): against autograd, central differences and torch's own formats; and what the entry points refuse."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import documents_ref as R
from step_gpt_train_gb300 import data, gpt2 as g

torch.manual_seed(1)


def table(rot, **kw):
    return torch.tensor([round(f * 2.0 ** 64) for f in R.turns(rot, **kw)], dtype=torch.int64)


@pytest.mark.parametrize("rot", [0, 2, 8, 64, 128])
@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "parts"])
def test_turns(rot, scaling):
    kw = dict(base=500.0, scaling=scaling, factor=4.0, context=2048, fast=32.0, slow=1.0)
    got, want = g.gpt2_rotary_turns(rot, **kw), R.turns(rot, **kw)
    assert got.shape == (rot // 2,)
    for a, b in zip(got.tolist(), want):  # pow against exp of log: a few units of 2^-53, the exponents up to log(500)
        assert abs(a / 2.0 ** 64 - b) <= 64 * 2.0 ** -53 * b


def test_stretched_turns_keep_and_divide():
    plain, parts, base = (R.turns(64, scaling=s, factor=8.0, context=8192) for s in ("plain", "parts", "base"))
    assert parts[0] == plain[0] and math.isclose(parts[-1], plain[-1] / 8)
    assert base[0] == plain[0] and math.isclose(base[-1], plain[-1] / 8, rel_tol=1e-12)
    assert all(a >= b for a, b in zip(parts, parts[1:]))


@pytest.mark.parametrize("bad", [dict(rot=7), dict(rot=-2), dict(base=1.0), dict(base=math.inf), dict(factor=0.5),
                                 dict(factor=math.nan), dict(scaling="parts", context=0.0),
                                 dict(scaling="parts", fast=1.0), dict(scaling="parts", slow=-1.0)])
def test_turns_refuses(bad):
    with pytest.raises(g.GPT2Error, match="GPT2_ERR_ARG"):
        g.gpt2_rotary_turns(**{"rot": 8, **bad})


def test_turns_refuses_a_name():
    with pytest.raises(ValueError):
        g.gpt2_rotary_turns(8, scaling="yarn-like")


def test_angles_wrap_exactly():
    t = table(8)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071]).int()
    cos, sin = R._cos_sin(pos, t)
    for i, p in enumerate(pos.tolist()):
        for j, x in enumerate(t.tolist()):
            a = (p * x % (1 << 64)) / 2.0 ** 64 * 2 * math.pi  # whole numbers until here
            assert abs(cos[i, 0, j] - math.cos(a)) < 1e-14 and abs(sin[i, 0, j] - math.sin(a)) < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [None, 1e-5])
def test_rotary_against_autograd(interleaved, eps):
    x = torch.randn(5, 3, 16, dtype=torch.float64, requires_grad=True)
    gamma = (1 + 0.3 * torch.randn(16, dtype=torch.float64)).requires_grad_()
    pos, t = torch.tensor([0, 1, 7, 100, -3]).int(), table(8)
    y, _ = R.rotary(x, pos, t, gamma, eps, interleaved, 1.2)
    # against complex products
    n = x if eps is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * gamma
    a, b = R._pairs(8, interleaved)
    c = torch.complex(n[..., a], n[..., b]) * torch.polar(
        torch.tensor(1.2, dtype=torch.float64), pos.double()[:, None, None] * (t.double() * 2.0 ** -64 * 2 * math.pi))
    assert torch.allclose(y[..., a], c.real, atol=1e-12) and torch.allclose(y[..., b], c.imag, atol=1e-12)
    assert torch.allclose(y[..., 8:], n[..., 8:], atol=1e-12)  # two forms of the root: a few units of 2^-53
    dy = torch.randn_like(y)
    (y * dy).sum().backward()
    dx, dgamma, _, _ = R.rotary_backward(dy, x.detach(), pos, t, gamma.detach(), eps, interleaved, 1.2)
    assert torch.allclose(dx, x.grad, atol=1e-12)
    assert (dgamma is None) == (eps is None)
    if eps is not None:
        assert torch.allclose(dgamma, gamma.grad, atol=1e-12)


def test_rotary_depends_on_distance_only():
    q, k, t = torch.randn(1, 1, 32).double(), torch.randn(1, 1, 32).double(), table(32)
    dot = lambda p: (R.rotary(q, torch.tensor([p]), t)[0] * R.rotary(k, torch.tensor([p + 9]), t)[0]).sum()  # noqa: E731
    assert abs(dot(0) - dot(1000)) < 1e-9


def test_classifier_against_autograd():
    x, w = torch.randn(6, 8, dtype=torch.float64, requires_grad=True), torch.randn(16, 8, dtype=torch.float64,
                                                                                 requires_grad=True)
    t = torch.tensor([0, 3, 10, 5, -1, 99]).int()
    losses, lse, _, _ = R.classifier(x, w, t, 11)
    tt = torch.tensor([0, 3, 10, 5, 0, 0])
    assert torch.allclose(losses, torch.nn.functional.cross_entropy(x @ w[:11].T, tt, reduction="none"), atol=1e-12)
    d, e = torch.rand(6, dtype=torch.float64), torch.randn(6, dtype=torch.float64)
    d[2] = e[2] = 0
    ((losses * d).sum() + (lse * e).sum()).backward()
    dx, dw, _, _ = R.classifier_backward(x.detach(), w.detach(), t, 11, d, e, torch.float32)
    assert torch.allclose(dx, x.grad, atol=1e-12) and torch.allclose(dw, w.grad[:11], atol=1e-12)
    assert not dx[2].any()


def test_classifier_gradient_against_differences():
    x, w, t = torch.randn(3, 8).double(), torch.randn(5, 8).double(), torch.tensor([1, 4, 0]).int()
    d = torch.tensor([0.3, 1.0, -0.5]).double()
    dx, _, _, _ = R.classifier_backward(x, w, t, 5, d, None, torch.float32)
    h = 1e-6
    for i, j in ((0, 0), (1, 3), (2, 7)):
        step = torch.zeros_like(x)
        step[i, j] = h
        up, down = ((R.classifier(x + s * step, w, t, 5)[0] * d).sum() for s in (1, -1))
        assert abs((up - down) / (2 * h) - dx[i, j]) < 1e-8


def test_draws_are_splitmix64():
    z = torch.tensor([0, 1, -1, 2 ** 62, -2 ** 63], dtype=torch.int64)
    want = data.splitmix64_mix(z.numpy().view(np.uint64))
    assert (R.mix(z).numpy().view(np.uint64) == want).all()
    assert [R.mix(int(x) & (1 << 64) - 1) for x in z.tolist()] == want.tolist()
    um, uv = R.draws(100001, 3, 7, 12345)
    assert um.shape == uv.shape == (100001,)
    for u in (um, uv):
        assert 0 <= u.min() and u.max() < 1 and abs(u.mean() - 0.5) < 5 / math.sqrt(12 * 100001)
    assert abs(torch.corrcoef(torch.stack((um, uv)))[0, 1]) < 5 / math.sqrt(100001)
    # a value's draw does not depend on the tensor's length
    assert torch.equal(R.draws(77, 3, 7, 12345)[0], um[:77])


def test_codes_of_the_first_moment_are_e4m3():
    code = torch.arange(256).to(torch.uint8)
    want = code.view(torch.float8_e4m3fn).float().double()
    got = R.values(code, torch.full((2,), 127, dtype=torch.uint8), "m")
    assert torch.equal(got.nan_to_num(7e9), want.nan_to_num(7e9))


def test_codes_of_the_second_moment_are_the_top_of_fp16():
    code = torch.arange(255).to(torch.uint8)
    want = (code.to(torch.int16) << 7).view(torch.float16).double()  # sign 0, 5 exponent bits, 3 of 10 mantissa bits
    got = R.values(code, torch.full((2,), 127, dtype=torch.uint8), "v")
    small = code < 248  # fp16's last exponent is infinity
    assert torch.equal(got[small], want[small])


@pytest.mark.parametrize("kind", ["m", "v"])
def test_rounding_is_right_on_average(kind):
    x = torch.exp(3 * torch.randn(256).double())
    if kind == "m":
        x = x * torch.sign(torch.randn(256))
    s = R.scales(x, kind)
    u = (torch.arange(65536).double() / 65536)[:, None]
    got = torch.stack([R.stored(x, s, r, kind) for r in u[::64]])
    # each of the 1024 equidistant u once: the mean is x to a 1024th of a step, which is an eighth of x's binade, or
    # the lowest code where x is below the lowest whole exponent
    unit = torch.exp2(s.double() - 127).repeat_interleave(128)
    lowest = unit * 2.0 ** (-9 if kind == "m" else -17)
    ok = (got.mean(0) - x).abs() <= torch.maximum(x.abs() / 8, lowest) / 1024
    floor = (x.abs() < lowest) & (kind == "v")  # kept above 0
    assert (ok | floor).all() and floor.sum() < 8
    # a value that a code stands for stays what it is
    once = R.stored(x, s, torch.full((256,), 0.999).double(), kind)
    assert torch.equal(R.stored(once, R.scales(x, kind), torch.zeros(256).double(), kind), once)


def test_adamw_is_torchs():
    p = torch.nn.Parameter(torch.randn(50, dtype=torch.float64))
    o = torch.optim.AdamW([p], lr=0.0078125, betas=(0.875, 0.96875), eps=2.0 ** -20, weight_decay=0.125)
    th, m, v = p.detach().clone(), torch.zeros(50).double(), torch.zeros(50).double()
    for t in (1, 2, 3):
        p.grad = torch.randn(50, dtype=torch.float64)
        o.step()
        th, m, v = R.adamw(th, p.grad, m, v, 0.0078125, 0.875, 0.96875, 2.0 ** -20, 0.125, t, 1.0)
    assert torch.allclose(th, p.detach(), atol=1e-12)


# ---------------------------------------------------------------- what the entry points refuse (no launch)

P = 1 << 20  # an aligned address that nothing reads


def rotary_args(**kw):
    c = dict(dtype=1, qo=P, qos=512, ko=P, kos=512, q=P, qs=512, k=P, ks=512, qg=P, kg=P, pos=P, turns=P, N=4, Hq=8,
             Hk=2, hd=64, rot=64, inter=0, norm=1, eps=1e-6, amp=1.0, stream=None)
    c.update(kw)
    return c


BAD_ROTARY = [dict(dtype=2), dict(N=-1), dict(Hq=-1), dict(Hq=0, Hk=0), dict(hd=24), dict(hd=256), dict(rot=72),
              dict(rot=4), dict(rot=-8), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
              dict(amp=math.inf), dict(q=None), dict(ko=None), dict(pos=None), dict(turns=None), dict(q=P + 8),
              dict(ko=P + 2), dict(qg=P + 4), dict(qs=500), dict(qs=504), dict(kos=120), dict(qos=1 << 31)]


@pytest.mark.parametrize("bad", BAD_ROTARY, ids=str)
def test_rotary_refuses(bad):
    lib = g.load_library(build=True)
    c = rotary_args(**bad)
    assert lib.gpt2_op_qk_norm_rotary_forward(*c.values()) == -1
    d = c
    back = (d["dtype"], d["qo"], d["qos"], d["ko"], d["kos"], P, P, d["q"], d["qs"], d["k"], d["ks"], d["q"], d["qs"],
            d["k"], d["ks"], d["qg"], d["kg"], d["pos"], d["turns"], d["N"], d["Hq"], d["Hk"], d["hd"], d["rot"],
            d["inter"], d["norm"], d["eps"], d["amp"], P, 1 << 30, None)
    assert lib.gpt2_op_qk_norm_rotary_backward(*back) == -1
    assert lib.gpt2_op_qk_norm_rotary_forward(*rotary_args(N=0).values()) == 0
    if d["N"] > 0 and bad == dict(dtype=2):
        good = (1, *back[1:-3], None, 0, None)
        assert lib.gpt2_op_qk_norm_rotary_backward(*good) == -7  # no scratch


@pytest.mark.parametrize("bad", [dict(dtype=7), dict(N=-1), dict(C=12), dict(C=0), dict(V=0), dict(losses=None),
                                 dict(lse=None), dict(x=None), dict(w=None), dict(targets=None), dict(x=P + 8),
                                 dict(w=P + 4), dict(N=1 << 28), dict(V=1 << 28), dict(N=(1 << 31) - 1, C=8), dict(N=1 << 27, V=1 << 27, C=8)], ids=str)
def test_classifier_refuses(bad):
    lib = g.load_library(build=True)
    c = dict(dtype=1, losses=P, lse=P, x=P, w=P, targets=P, N=4, C=64, V=50)
    c.update(bad)
    assert lib.gpt2_op_linear_classifier_forward(*c.values(), P, 1 << 40, None, None) == -1
    bad_back = {k: v for k, v in c.items() if k not in ("losses",)}
    a = (bad_back["dtype"], P, P, 1, 0, c["x"], c["w"], c["targets"], c["lse"], P, None, c["N"], c["C"], c["V"],
         max(8, (c["V"] + 7) // 8 * 8), P, 1 << 40, None, None)
    if "losses" not in bad:
        assert lib.gpt2_op_linear_classifier_backward(*a) == -1


def test_classifier_backward_refuses():
    lib = g.load_library(build=True)

    def call(dtype=1, dx=P, dw=P, dw32=1, acc=0, V=50, Vp=56, N=4, scratch=P, nb=1 << 40):
        return lib.gpt2_op_linear_classifier_backward(dtype, dx, dw, dw32, acc, P, P, P, P, P, None, N, 64, V, Vp,
                                                      scratch, nb, None, None)
    assert call(Vp=48) == call(Vp=52) == call(dw32=0, acc=1) == call(dtype=0, dw32=0) == -1
    assert call(dx=None) == call(dw=None) == call(dx=P + 8) == call(dw=P + 2) == -1
    assert call(scratch=None) == call(nb=100) == -7
    assert lib.gpt2_op_linear_classifier_forward(1, P, P, P, P, P, 4, 64, 50, None, 0, None, None) == -7
    assert lib.gpt2_op_linear_classifier_forward(1, None, None, None, None, None, 0, 64, 50, None, 0, None, None) == 0


def entry(**kw):
    c = dict(master=P, param_bf16=P, grad=P, m=P, v=P, m_scale=P, v_scale=P, n=100, weight_decay=0.1)
    c.update(kw)
    return g.gpt2_adamw_tensor(**c)


@pytest.mark.parametrize("bad", [dict(master=None), dict(grad=None), dict(m=None), dict(v=None), dict(master=P + 2),
                                 dict(grad=P + 2), dict(m=P + 1), dict(param_bf16=P + 1), dict(n=-1),
                                 dict(n=1 << 43)], ids=str)
def test_adamw_refuses_a_tensor(bad):
    lib = g.load_library(build=True)
    a = (g.gpt2_adamw_tensor * 2)(entry(n=0, master=None), entry(**bad))
    assert lib.gpt2_op_adamw_many(a, 2, 0, 32, 1e-3, 0.9, 0.95, 1e-8, 1.0, 0.0, None, 1, 0, None, 0, None) == -1


def test_adamw_refuses():
    lib = g.load_library(build=True)
    a = (g.gpt2_adamw_tensor * 1)(entry())

    def call(array=a, n=1, dtype=0, bits=32, b1=0.9, b2=0.95, eps=1e-8, clip=0.0, norm=None, t=1, sc=None, nb=0):
        return lib.gpt2_op_adamw_many(array, n, dtype, bits, 1e-3, b1, b2, eps, 1.0, clip, norm, t, 0, sc, nb, None)
    nan = math.nan
    for kw in (dict(array=None), dict(n=-1), dict(dtype=3), dict(bits=16), dict(b1=1.0), dict(b2=1.0), dict(b1=-0.1),
               dict(b2=nan), dict(eps=-1.0), dict(eps=nan), dict(clip=-1.0), dict(clip=nan), dict(t=0)):
        assert call(**kw) == -1, kw
    assert call(clip=1.0) == call(norm=P) == call(clip=1.0, sc=P, nb=8) == -7
    assert call(n=0) == 0 and call(array=None, n=0) == 0
    for kw in (dict(m_scale=None), dict(v_scale=None)):
        assert call((g.gpt2_adamw_tensor * 1)(entry(**kw)), bits=8) == -1
    ptr = (ctypes.c_void_p * 1)(P)
    none = (ctypes.c_void_p * 1)(None)
    odd = (ctypes.c_void_p * 1)(P + 1)
    states = lambda m, v, dtype=1, x=a: lib.gpt2_op_adamw_many_states(x, m, v, 1, dtype, None)  # noqa: E731
    assert states(none, ptr) == states(ptr, none) == states(odd, ptr) == states(ptr, ptr, 5) == states(None, ptr) == -1
