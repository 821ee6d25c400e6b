"""Head norms with rotary positions, the cross entropy of hidden states and AdamW over many tensors: what the host
side holds, hands on and refuses (CPU; nothing is launched)."""
import decimal
import gc
import os
import subprocess
import sys
import weakref

import numpy as np
import pytest
import torch

from step_gpt_train_gb300 import gpt2 as g

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    return g.load_library(build=True)


def tensors(bits=32, sizes=(5, 300)):
    """Columns of a list of tensors, each on memory of its own."""
    z = lambda dtype, per=1: [torch.zeros(-(-n // per), dtype=dtype) for n in sizes]  # noqa: E731
    moment = F32 if bits == 32 else torch.uint8
    c = dict(masters=z(F32), grads=z(F32), ms=z(moment), vs=z(moment), params=z(BF))
    if bits == 8:
        c |= dict(m_scales=z(torch.uint8, 128), v_scales=z(torch.uint8, 128), m_values=z(F32), v_values=z(F32))
    return c


# ---------------------------------------------------------------- the list of AdamW over many tensors

@pytest.mark.parametrize("bits", [32, 8])
def test_a_list_keeps_the_memory_it_was_given(bits):
    """Tensors that get other memory (`.data`, as Module.to sets it) leave the old one to the list: a step would write
    to it."""
    c, alive = tensors(bits), []
    for xs in c.values():
        for i, x in enumerate(xs):
            if x.dtype is BF:
                continue  # (numpy has no such type)
            a = np.zeros(x.numel(), dtype=x.numpy().dtype)
            alive.append(weakref.ref(a))
            xs[i] = torch.from_numpy(a)
    del a
    h = g.gpt2_adamw_tensors(**c)
    address = h.array[1].master
    assert address == c["masters"][1].data_ptr()
    for xs in c.values():
        for x in xs:
            x.data = torch.zeros_like(x)
    gc.collect()
    assert c["masters"][1].data_ptr() != address and all(r() is not None for r in alive)
    del h
    gc.collect()
    assert all(r() is None for r in alive)


def leaves(sizes=(5, 300)):
    """Parameters whose gradients stand in their .grad."""
    c = tensors(32, sizes)
    c["masters"] = [torch.nn.Parameter(x) for x in c["masters"]]
    for p, x in zip(c["masters"], c["grads"]):
        p.grad = x
    return c


STEP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, t=1)


def test_a_step_refuses_gradients_that_are_no_longer_the_parameters():
    c = leaves()
    h = g.gpt2_adamw_tensors(**c)
    with pytest.raises(RuntimeError, match="current CUDA device"):  # all is well but the device
        g.gpt2_op_adamw_many(h, **STEP)
    c["masters"][1].grad = None  # as zero_grad leaves it
    with pytest.raises(RuntimeError, match="give this step's grads"):
        g.gpt2_op_adamw_many(h, **STEP)
    c["masters"][1].grad = torch.zeros(300)  # as the next backward pass does
    with pytest.raises(RuntimeError, match="give this step's grads"):
        g.gpt2_op_adamw_many(h, **STEP)
    c["masters"][1].grad = c["grads"][1]
    with pytest.raises(RuntimeError, match="current CUDA device"):
        g.gpt2_op_adamw_many(h, **STEP)
    # bf16 parameters, their gradients beside fp32 masters
    c = tensors(32)
    c["params"] = [torch.nn.Parameter(x) for x in c["params"]]
    c["grads"] = [x.to(BF) for x in c["grads"]]
    for p, x in zip(c["params"], c["grads"]):
        p.grad = x
    h = g.gpt2_adamw_tensors(**c)
    c["params"][0].grad = torch.zeros(5, dtype=BF)
    with pytest.raises(RuntimeError, match="give this step's grads"):
        g.gpt2_op_adamw_many(h, **STEP)


@pytest.mark.parametrize("bad", [[torch.zeros(5)], [torch.zeros(5), torch.zeros(299)], [torch.zeros(5), None],
                                 [torch.zeros(5), torch.zeros(300, dtype=BF)], [torch.zeros(5), torch.zeros(600)[::2]]],
                         ids=["one", "short", "missing", "bf16", "strided"])
def test_a_step_refuses_new_gradients_that_do_not_fit(bad):
    h = g.gpt2_adamw_tensors(**tensors())
    before = [h.array[i].grad for i in range(2)]
    with pytest.raises(ValueError, match="grads"):
        g.gpt2_op_adamw_many(h, **STEP, grads=bad)
    with pytest.raises(RuntimeError, match="current CUDA device"):
        g.gpt2_op_adamw_many(h, **STEP, grads=[torch.zeros(5), torch.zeros(300)])
    assert [h.array[i].grad for i in range(2)] == before  # what is refused leaves the list as it was


@pytest.mark.parametrize("bits", [32, 8])
def test_a_list_refuses_tensors_that_overlap(bits):
    c = tensors(bits, (300, 5, 300))
    g.gpt2_adamw_tensors(**c)
    for k in c:
        twice = dict(c)
        twice[k] = [c[k][0], c[k][1], c[k][0]]
        if k == "grads":  # which are only read
            g.gpt2_adamw_tensors(**twice)
            continue
        with pytest.raises(ValueError, match="overlap"):
            g.gpt2_adamw_tensors(**twice)
    # in part; across columns; one behind the other is no overlap, nor are tensors without values
    flat = torch.zeros(605)
    for parts in ([flat[:300], flat[300:305], flat[304:604]], [flat[:300], c["ms"][0][:5].float(), flat[299:599]]):
        with pytest.raises(ValueError, match="overlap"):
            g.gpt2_adamw_tensors(**{**c, "masters": parts})
    g.gpt2_adamw_tensors(**{**c, "masters": [flat[:300], flat[300:305], flat[305:]]})
    if bits == 32:
        with pytest.raises(ValueError, match="overlap"):
            g.gpt2_adamw_tensors(**{**c, "vs": c["ms"]})
    none = [torch.zeros(0)] * 2
    g.gpt2_adamw_tensors(none, none, none, none)


def test_moments_of_an_empty_list_are_read_back():
    h = g.gpt2_adamw_tensors([], [], [], [], m_scales=[], v_scales=[], m_values=[], v_values=[])
    g.gpt2_op_adamw_many(h, **STEP)
    g.gpt2_op_adamw_many_states(h)
    with pytest.raises(ValueError):  # there is no place for values
        g.gpt2_op_adamw_many_states(g.gpt2_adamw_tensors([], [], [], []))


# ---------------------------------------------------------------- scratch of the loss's gradient

@pytest.mark.parametrize("mode,size", [(1, 2), (0, 4)])
@pytest.mark.parametrize("N,C,V,Vp", [((1 << 27) + 5, 8, 15, 16), (1 << 20, 64, 100, 104), (1000, 64, 300, 304),
                                      (4096, 768, 50257, 50304)])
def test_scratch_of_a_small_vocabulary_is_no_wider_than_it(lib, mode, size, N, C, V, Vp):
    """One piece of dz: its columns are dw's rows, not the next 256."""
    got = lib.gpt2_op_linear_classifier_backward_scratch(mode, N, C, V, Vp, 0)
    # besides dz: the scale, and the parts of products split at most 64 times along k (fp32: as many as fill the device)
    parts = 64 * 4 * max(128 * 256, -(-Vp // 128) * 128 * -(-C // 128) * 128)
    assert N * Vp * size <= got <= N * Vp * size + 1024 + parts

@pytest.mark.parametrize("mode,size", [(1, 2), (0, 4)])
@pytest.mark.parametrize("N,C,V,Vp", [(32768, 768, 50257, 50304), (70000, 1024, 50257, 50264), (32768, 128, 20001, 20008)])
def test_scratch_of_several_pieces(mode, size, N, C, V, Vp):
    """Equal pieces, as few as 1 GB each asks for, on a host without a GPU too (in a process of its own: the call
    divided by the number of SM pairs there, which is 0)."""
    ask = ("from step_gpt_train_gb300 import gpt2 as g; "
           f"print(g.load_library().gpt2_op_linear_classifier_backward_scratch({mode}, {N}, {C}, {V}, {Vp}, 0))")
    r = subprocess.run([sys.executable, "-c", ask], capture_output=True, text=True, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""},
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
    pieces = -(-V // ((1 << 30) // (N * size) // 256 * 256))  # (of whole tiles of 256)
    wide = -(-V // pieces)  # (a piece's columns: that, rounded up to whole tiles)
    rest = N * C * 4 * (mode == 1) + 64 * 4 * (wide + 256) * (C + 128) + 1024  # dx in fp32; parts of products
    assert N * wide * size <= int(r.stdout) <= N * (wide + 255) * size + rest


# ---------------------------------------------------------------- turns

def decimal_turns(rot, base, scaling, factor, context, fast, slow):
    """2^64 times the fractions of a turn, to 60 digits."""
    D = decimal.Decimal
    with decimal.localcontext() as c:
        c.prec = 60
        # pi: Machin's formula
        atan = lambda n: sum((-1) ** k / (D(n) ** (2 * k + 1) * (2 * k + 1)) for k in range(60))  # noqa: E731
        pi = 4 * (4 * atan(5) - atan(239))
        base, factor, context, fast, slow = (D(x) for x in (base, factor, context, fast, slow))
        log = base.ln()
        if scaling == "base" and rot > 2:
            log += factor.ln() * rot / (rot - 2)
        out = []
        for j in range(rot // 2):
            f = (log * (-2 * j) / rot).exp() / (2 * pi)
            if scaling == "linear":
                f /= factor
            if scaling == "parts":
                keep = min(D(1), max(D(0), (f * context - slow) / (fast - slow)))
                f *= keep + (1 - keep) / factor
            out.append(f * 2 ** 64)
        return out


@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "parts"])
@pytest.mark.parametrize("rot,base,factor", [(2, 1e4, 8.0), (8, 1e4, 1.0), (64, 1e4, 8.0), (128, 5e5, 32.0), (128, 1e6, 3.7),
                                             (64, 1.0000001, 1.5), (64, 1.7e308, 1e300)])
def test_turns_are_whole_to_their_last_bit(scaling, rot, base, factor):
    """turns[j] is the nearest whole number of 2^-64 turns: a position of 31 bits keeps its angle to 2^-34 of a turn."""
    kw = dict(base=base, scaling=scaling, factor=factor, context=8192.0, fast=32.0, slow=1.0)
    got, want = g.gpt2_rotary_turns(rot, **kw).tolist(), decimal_turns(rot, **kw)
    # half a unit of the rounding, and 2^-20 of one for the arithmetic before it (two numbers of 53 bits each)
    assert all(abs(a - b) <= 0.5 + 2.0 ** -20 for a, b in zip(got, want)), max(abs(a - b) for a, b in zip(got, want))


@pytest.mark.parametrize("context,fast,slow", [(1e308, 32.0, 1.0), (1e308, 1.0, 1.0 - 2.0 ** -53), (1.0, 5e-324, 0.0),
                                               (1.0, 1e308, 0.0), (1e308, 1.5e307, 1e307), (1e6, 2.0 ** -1000, 0.0)])
def test_turns_of_any_borders(context, fast, slow):
    kw = dict(base=1e4, scaling="parts", factor=8.0, context=context, fast=fast, slow=slow)
    got, want = g.gpt2_rotary_turns(64, **kw).tolist(), decimal_turns(64, **kw)
    assert all(abs(a - b) <= 0.5 + 2.0 ** -20 for a, b in zip(got, want))
