"""Head norms with rotary positions, the cross entropy of hidden states and AdamW over many tensors on the GPU where
they are easily wrong, against the definitions in 64 bits."""
import math

import pytest
import torch

from oracle import documents_ref as R
from step_gpt_train_gb300 import gpt2 as g

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def seed():
    torch.manual_seed(12)
    torch.cuda.set_device(0)


def rnd(*shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, device="cuda") * std).to(dtype)


# ---------------------------------------------------------------- AdamW over many tensors

@pytest.mark.parametrize("grads", [F32, BF])
def test_adamw_many_takes_each_steps_gradients(grads):
    """Gradients that are new tensors in every step, given to one list, do what a new list for each step does."""
    sizes, hp = [5000, 77, 0, 40000], dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, max_grad_norm=0.5)
    one = {"masters": [rnd(n) for n in sizes], "params": [rnd(n).to(BF) for n in sizes],
           "ms": [torch.zeros(n, device="cuda") for n in sizes], "vs": [torch.zeros(n, device="cuda") for n in sizes]}
    two = {k: [x.clone() for x in v] for k, v in one.items()}
    h = g.gpt2_adamw_tensors(**one, grads=[torch.full((n,), math.nan, device="cuda").to(grads) for n in sizes])
    for t in (1, 2, 3):
        new = [rnd(n, dtype=grads) for n in sizes]
        g.gpt2_op_adamw_many(h, **hp, t=t, grads=new)
        g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**two, grads=new), **hp, t=t)
        for k in one:
            assert all(torch.equal(a, b) for a, b in zip(one[k], two[k])), (k, t)
    # the last ones stay the list's
    g.gpt2_op_adamw_many(h, **hp, t=4)
    g.gpt2_op_adamw_many(g.gpt2_adamw_tensors(**two, grads=new), **hp, t=4)
    assert all(torch.equal(a, b) for k in one for a, b in zip(one[k], two[k]))


def test_adamw_many_follows_a_backward_pass():
    """A loop that drops its gradients before each backward pass, as torch's zero_grad does."""
    p = torch.nn.Parameter(rnd(300))
    x = rnd(300)
    m, v = torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda")
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)
    (p * x).sum().backward()
    h = g.gpt2_adamw_tensors([p], [p.grad], [m], [v])
    want, wm, wv = p.detach().double(), m.double(), v.double()
    for t in (1, 2, 3):
        p.grad = None
        (p * p * x).sum().backward()
        want, wm, wv = R.adamw(want, p.grad.double(), wm, wv, wd=0.0, t=t, factor=1.0, lr=hp["lr"], b1=hp["beta1"],
                               b2=hp["beta2"], eps=hp["eps"])
        with pytest.raises(RuntimeError, match="give this step's grads"):
            g.gpt2_op_adamw_many(h, **hp, t=t)
        g.gpt2_op_adamw_many(h, **hp, t=t, grads=[p.grad])
        # a step is at most lr (1 - b1) / sqrt(1 - b2) of 1, in about 60 operations of U each
        assert ((p.detach().double() - want).abs() <= 64 * R.U * t * (want.abs() + hp["lr"])).all()
        want = p.detach().double()
        wm, wv = m.double(), v.double()
        g.gpt2_op_adamw_many(h, **{**hp, "lr": 0.0}, t=t)  # the gradients given stand in .grad: no refusal
        m.copy_(wm), v.copy_(wv)
    # gradients that are not the .grad are taken as they are, and stay the list's
    p.grad = None
    x = x.clone()
    g.gpt2_op_adamw_many(h, **hp, t=4, grads=[x])
    g.gpt2_op_adamw_many(h, **hp, t=5)


def test_adamw_many_lets_go_of_gradients_that_were_replaced():
    n, hp = 1 << 22, dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)
    p, m, v = (torch.nn.Parameter(rnd(n)), *(torch.zeros(n, device="cuda") for _ in range(2)))
    p.grad = rnd(n)
    h = g.gpt2_adamw_tensors([p], [p.grad], [m], [v])
    held = torch.cuda.memory_allocated()
    for t in (1, 2, 3):
        p.grad = rnd(n)
        g.gpt2_op_adamw_many(h, **hp, t=t, grads=[p.grad])
        assert torch.cuda.memory_allocated() == held


# ---------------------------------------------------------------- rotation

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [8, 64])
def test_angles_keep_their_bits_at_any_position(interleaved, rot):
    """Rotations of (1, 0) and (0, 1): cos and sin themselves, of all int32 positions."""
    n = 5000
    pos = torch.randint(-(1 << 31), 1 << 31, (n,), device="cuda").int()
    pos[:8] = torch.tensor([0, 1, -1, 2, 131071, 1 << 24, (1 << 31) - 1, -(1 << 31)]).int()
    turns = g.gpt2_rotary_turns(rot).cuda()
    a, b = (i.cuda() for i in R._pairs(rot, interleaved))
    q, k = torch.zeros(n, 1, 64, device="cuda"), torch.zeros(n, 1, 64, device="cuda")
    q[..., a] = 1
    k[..., b] = 1
    g.gpt2_op_qk_norm_rotary_forward(q, k, q, k, pos, turns, interleaved=interleaved)
    cos, sin = R._cos_sin(pos, turns)
    # the angle is taken off its nearest quarter turn before it becomes an fp32 number: at most an eighth of a turn is
    # left, a quarter of half a turn, whose rounding is 2^-27 of half a turn; then one unit of the last place (2^-23 at
    # most) of cos and sin
    for got, want, slope in ((q[..., a], cos, sin), (q[..., b], sin, cos), (k[..., a], -sin, cos), (k[..., b], cos, sin)):
        far = (got.double() - want).abs() - (math.pi * 2.0 ** -27 * slope.abs() + 2.0 ** -23 * want.abs() + 2.0 ** -50)
        assert (far <= 0).all(), far.max().item()
    assert not q[..., rot:].any() and not k[..., rot:].any()
    # back again: the transposed rotation
    ones, none = torch.zeros_like(q), torch.zeros_like(q)
    ones[..., a] = 1
    g.gpt2_op_qk_norm_rotary_backward(ones, none, ones, none, q, k, pos, turns, interleaved=interleaved)
    for got, want, slope in ((ones[..., a], cos, sin), (ones[..., b], -sin, cos)):
        assert ((got.double() - want).abs() <= math.pi * 2.0 ** -27 * slope.abs() + 2.0 ** -23 * want.abs() + 2.0 ** -50).all()

# ---------------------------------------------------------------- cross entropy of hidden states

@pytest.mark.parametrize("dtype", [BF, F32])
def test_probabilities_of_far_logits_are_off_by_lses_own_rounding_only(dtype):
    """Rows whose logits lie at 1.3e5 to 2.6e5, exact in fp32, with an lse that is exact too: p is exp(z - lse)."""
    n, C, V = 128, 16, 8
    x = torch.zeros(n, C, device="cuda", dtype=dtype)
    w = torch.zeros(V, C, device="cuda", dtype=dtype)
    x[:, 0] = 256 + 2 * torch.arange(n, device="cuda").to(dtype)  # eight bits: a bf16 number
    x[:, 1] = 1
    w[:, 0] = 512
    w[:, 1] = -0.25 * torch.arange(V, device="cuda").to(dtype)
    w[:, 8:] = torch.eye(V, device="cuda").to(dtype)  # dx's last columns are dz's
    lse = 512 * x[:, 0].float()
    t = torch.zeros(n, device="cuda", dtype=torch.int32)
    dx, dw = torch.empty_like(x), torch.empty(V, C, device="cuda")
    g.gpt2_op_linear_classifier_backward(dx, dw, x, w, t, lse, V, dlse=torch.ones(n, device="cuda"))
    p = torch.exp(w[:, 1].double()).expand(n, V)
    # dz is rounded to its type and dx keeps it; before that: z - lse is exact in fp32 and at most 1.75, log2 e and its
    # product are off by 2^-23 of it, the exponentials by 2^-22 each, two products by 2^-24 each
    assert ((dx[:, 8:].double() - p).abs() <= p * (R.HALF[dtype] + 2.0 ** -20)).all()
