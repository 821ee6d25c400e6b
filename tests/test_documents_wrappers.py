"""What the wrappers of head norms with rotary positions, the cross entropy of hidden states and AdamW over many
tensors refuse before they hand addresses to a kernel (CPU; nothing is launched)."""
import pytest
import torch

from step_gpt_train_gb300 import gpt2 as g

BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    return g.load_library(build=True)


def rotary(dtype=BF, **kw):
    c = dict(q=torch.zeros(4, 2, 64, dtype=dtype), k=torch.zeros(4, 1, 64, dtype=dtype), pos=torch.zeros(4).int(),
             turns=torch.zeros(32).long(), q_gamma=torch.ones(64, dtype=dtype), k_gamma=torch.ones(64, dtype=dtype),
             dq_gamma=torch.ones(64), dk_gamma=torch.ones(64), eps=1e-6)
    c.update(kw)
    for n in ("qo", "dqo", "dq"):
        c.setdefault(n, torch.zeros_like(c["q"]))
    for n in ("ko", "dko", "dk"):
        c.setdefault(n, torch.zeros_like(c["k"]))
    rest = [c["q"], c["k"], c["pos"], c["turns"]]
    kw = {n: c[n] for n in ("q_gamma", "k_gamma", "eps")}
    return [c["qo"], c["ko"]] + rest, kw, [c["dq"], c["dk"], c["dqo"], c["dko"]] + rest, \
        {**kw, "dq_gamma": c["dq_gamma"], "dk_gamma": c["dk_gamma"]}


BAD_ROTARY = {
    "float16": lambda: rotary(F16),
    "int32": lambda: rotary(torch.int32, q_gamma=None, k_gamma=None),
    "two dimensions": lambda: rotary(q=torch.zeros(4, 128, dtype=BF)),
    "k of other rows": lambda: rotary(k=torch.zeros(5, 1, 64, dtype=BF)),
    "k of another head size": lambda: rotary(k=torch.zeros(4, 1, 32, dtype=BF)),
    "k of another type": lambda: rotary(k=torch.zeros(4, 1, 64)),
    "qo of another shape": lambda: rotary(qo=torch.zeros(4, 1, 64, dtype=BF), dq=torch.zeros(4, 1, 64, dtype=BF)),
    "heads apart": lambda: rotary(q=torch.zeros(4, 2, 128, dtype=BF)[..., :64]),
    "values apart": lambda: rotary(q=torch.zeros(4, 2, 128, dtype=BF)[..., ::2]),
    "int64 positions": lambda: rotary(pos=torch.zeros(4).long()),
    "few positions": lambda: rotary(pos=torch.zeros(3).int()),
    "positions, every other one": lambda: rotary(pos=torch.zeros(8).int()[::2]),
    "float turns": lambda: rotary(turns=torch.zeros(32)),
    "turns of two dimensions": lambda: rotary(turns=torch.zeros(4, 8).long()),
    "fp32 gamma of bf16 heads": lambda: rotary(q_gamma=torch.ones(64)),
    "short gamma": lambda: rotary(k_gamma=torch.ones(32, dtype=BF)),
}


@pytest.mark.parametrize("name", BAD_ROTARY)
def test_rotary_refuses(name):
    forward, kf, backward, kb = BAD_ROTARY[name]()
    with pytest.raises(ValueError):
        g.gpt2_op_qk_norm_rotary_forward(*forward, **kf)
    with pytest.raises(ValueError):
        g.gpt2_op_qk_norm_rotary_backward(*backward, **kb)


@pytest.mark.parametrize("bad", [dict(dq_gamma=torch.ones(64, dtype=BF)), dict(dk_gamma=torch.ones(32)),
                                 dict(dq_gamma=torch.ones(128)[::2]), dict(eps=None),
                                 dict(dqo=torch.zeros(4, 2, 32, dtype=BF))])
def test_rotary_backward_refuses(bad):
    _, _, a, kw = rotary(**bad)
    with pytest.raises(ValueError):
        g.gpt2_op_qk_norm_rotary_backward(*a, **kw)


def test_rotary_refuses_tensors_that_are_not_on_the_device():
    forward, kf, backward, kb = rotary()
    with pytest.raises(RuntimeError, match="current CUDA device"):
        g.gpt2_op_qk_norm_rotary_forward(*forward, **kf)
    with pytest.raises(RuntimeError, match="current CUDA device"):
        g.gpt2_op_qk_norm_rotary_backward(*backward, **kb)


def classifier(dtype=BF, V=50, **kw):
    c = dict(losses=torch.zeros(4), lse=torch.zeros(4), x=torch.zeros(4, 64, dtype=dtype),
             w=torch.zeros(56, 64, dtype=dtype), targets=torch.zeros(4).int(), dloss=torch.zeros(4), dlse=torch.zeros(4),
             accumulate=False, status=None)
    c.update(kw)
    c.setdefault("dx", torch.zeros_like(c["x"]))
    c.setdefault("dw", torch.zeros_like(c["w"]))
    return [c[n] for n in ("losses", "lse", "x", "w", "targets")] + [V], dict(status=c["status"]), \
        [c[n] for n in ("dx", "dw", "x", "w", "targets", "lse")] + [V], \
        {n: c[n] for n in ("dloss", "dlse", "accumulate", "status")}


BOTH = {
    "float16": lambda: classifier(F16),
    "float64": lambda: classifier(torch.float64),
    "w of another type": lambda: classifier(w=torch.zeros(56, 64)),
    "w of another width": lambda: classifier(w=torch.zeros(56, 32, dtype=BF)),
    "w transposed": lambda: classifier(w=torch.zeros(64, 56, dtype=BF).T),
    "x, every other row": lambda: classifier(x=torch.zeros(8, 64, dtype=BF)[::2]),
    "x of three dimensions": lambda: classifier(x=torch.zeros(2, 2, 64, dtype=BF)),
    "more tokens than rows of w": lambda: classifier(V=57),
    "no tokens": lambda: classifier(V=0),
    "int64 targets": lambda: classifier(targets=torch.zeros(4).long()),
    "few targets": lambda: classifier(targets=torch.zeros(3).int()),
    "bf16 lse": lambda: classifier(lse=torch.zeros(4, dtype=BF)),
    "few lse": lambda: classifier(lse=torch.zeros(3)),
}


@pytest.mark.parametrize("name", BOTH)
def test_classifier_refuses(name):
    forward, kf, backward, kb = BOTH[name]()
    with pytest.raises(ValueError):
        g.gpt2_op_linear_classifier_forward(*forward, **kf)
    with pytest.raises(ValueError):
        g.gpt2_op_linear_classifier_backward(*backward, **kb)


@pytest.mark.parametrize("bad", [dict(dx=torch.zeros(4, 64)), dict(dx=torch.zeros(4, 32, dtype=BF)),
                                 dict(dw=torch.zeros(50, 64, dtype=BF)), dict(dw=torch.zeros(56, 64, dtype=F16)),
                                 dict(dw=torch.zeros(64, 56).T), dict(accumulate=True), dict(dloss=torch.zeros(3)),
                                 dict(dlse=torch.zeros(4, dtype=BF)), dict(dloss=torch.zeros(8)[::2]),
                                 dict(dtype=F32, dw=torch.zeros(56, 64, dtype=BF))], ids=str)
def test_classifier_backward_refuses(bad):
    _, _, a, kw = classifier(**bad)
    with pytest.raises(ValueError):
        g.gpt2_op_linear_classifier_backward(*a, **kw)


def test_classifier_refuses_tensors_that_are_not_on_the_device():
    for status in (None, torch.zeros(1).int()):
        forward, kf, backward, kb = classifier(status=status)
        with pytest.raises(RuntimeError, match="current CUDA device"):
            g.gpt2_op_linear_classifier_forward(*forward, **kf)
        with pytest.raises(RuntimeError, match="current CUDA device"):
            g.gpt2_op_linear_classifier_backward(*backward, **kb)


def tensors(bits=8, **kw):
    n = (5, 300)
    c = dict(masters=[torch.zeros(x) for x in n], grads=[torch.zeros(x) for x in n],
             ms=[torch.zeros(x) if bits == 32 else torch.zeros(x).byte() for x in n],
             vs=[torch.zeros(x) if bits == 32 else torch.zeros(x).byte() for x in n],
             params=[torch.zeros(x, dtype=BF) for x in n])
    if bits == 8:
        c |= {k: [torch.zeros(-(-x // 128)).byte() for x in n] for k in ("m_scales", "v_scales")}
    return c | kw


def test_tensors_are_taken():
    for bits in (8, 32):
        h = g.gpt2_adamw_tensors(**tensors(bits), weight_decay=[0.1, 0.0])
        assert (h.bits, h.count, h.array[1].n) == (bits, 2, 300) and h.array[0].weight_decay == pytest.approx(0.1)
    h = g.gpt2_adamw_tensors(**tensors(8, params=[None, torch.zeros(300, dtype=BF)]))
    assert h.array[0].param_bf16 is None and h.array[1].param_bf16
    two = torch.zeros(2, 150)  # any shape
    assert g.gpt2_adamw_tensors(**tensors(32, masters=[torch.zeros(5), two])).array[1].master == two.data_ptr()
    assert g.gpt2_adamw_tensors([], [], [], []).count == 0


BAD_TENSORS = {
    "one gradient": lambda t: t.update(grads=t["grads"][:1]),
    "decay of one": lambda t: t.update(weight_decay=[0.1]),
    "a gradient missing": lambda t: t.update(grads=[t["grads"][0], None]),
    "a moment missing": lambda t: t.update(ms=[t["ms"][0], None]),
    "a scale missing": lambda t: t.update(m_scales=[t["m_scales"][0], None]),
    "no scales": lambda t: t.update(v_scales=None),
    "few scales": lambda t: t.update(v_scales=[torch.zeros(1).byte()] * 2),
    "short gradient": lambda t: t.update(grads=[torch.zeros(5), torch.zeros(299)]),
    "mixed gradients": lambda t: t.update(grads=[torch.zeros(5), torch.zeros(300, dtype=BF)]),
    "mixed moments": lambda t: t.update(vs=[torch.zeros(5), torch.zeros(300)]),
    "float16 gradients": lambda t: t.update(grads=[x.half() for x in t["grads"]]),
    "bf16 masters": lambda t: t.update(masters=[x.to(BF) for x in t["masters"]]),
    "fp32 copies": lambda t: t.update(params=[x.float() for x in t["params"]]),
    "a strided master": lambda t: t.update(masters=[torch.zeros(10)[::2], torch.zeros(300)]),
    "int8 moments": lambda t: t.update(ms=[x.char() for x in t["ms"]]),
    "values of one moment": lambda t: t.update(m_values=[torch.zeros(5), torch.zeros(300)]),
    "short values": lambda t: t.update(m_values=[torch.zeros(5)] * 2, v_values=[torch.zeros(5), torch.zeros(300)]),
    "a value missing": lambda t: t.update(m_values=[torch.zeros(5), None], v_values=[torch.zeros(5), torch.zeros(300)]),
}


@pytest.mark.parametrize("name", BAD_TENSORS)
def test_tensors_refuses(name):
    t = tensors()
    BAD_TENSORS[name](t)
    with pytest.raises(ValueError):
        g.gpt2_adamw_tensors(**t)


def test_adamw_refuses():
    h = g.gpt2_adamw_tensors(**tensors())
    for kw in (dict(), dict(grad_norm=torch.zeros(1))):
        with pytest.raises(RuntimeError, match="current CUDA device"):
            g.gpt2_op_adamw_many(h, 1e-3, 0.9, 0.95, 1e-8, 1, **kw)
    with pytest.raises(ValueError):
        g.gpt2_op_adamw_many_states(h)
    with pytest.raises(ValueError):
        g.gpt2_op_adamw_many_states(g.gpt2_adamw_tensors(**tensors(32)))
    with pytest.raises(ValueError):
        g.gpt2_adamw_tensors(**tensors(32), m_values=[torch.zeros(5)] * 2, v_values=[torch.zeros(5)] * 2)
