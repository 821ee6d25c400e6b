"""What the wrappers of packed attention and token log-probabilities refuse before they hand addresses to a kernel:
types that the kernels do not read, layouts that they do not follow, arrays that are too short, tensors that are not
on the device (CPU; nothing is launched)."""
import pytest
import torch

from step_gpt_train_gb300 import gpt2 as g


@pytest.fixture(scope="module", autouse=True)
def lib():
    return g.load_library(build=True)


BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16


def attention(dtype=BF, **kw):
    """The operands of a call in order: forward's, backward's."""
    c = dict(q=torch.zeros(4, 2, 64, dtype=dtype), k=torch.zeros(9, 1, 64, dtype=dtype), lse=torch.zeros(2, 4),
             cu_q=torch.tensor([0, 1, 4]).int(), cu_k=torch.tensor([0, 3, 9]).int(), status=None)
    c.update(kw)
    for n in ("o", "dout", "dq"):
        c.setdefault(n, torch.zeros_like(c["q"]))
    for n in ("v", "dk", "dv"):
        c.setdefault(n, torch.zeros_like(c["k"]))
    tail = [c["cu_q"], c["cu_k"], 3, 6]
    return ([c[n] for n in ("o", "lse", "q", "k", "v")] + tail,
            [c[n] for n in ("dq", "dk", "dv", "dout", "q", "k", "v", "o", "lse")] + tail, dict(status=c["status"]))


BAD_ATTENTION = {
    "float16 operands": lambda: attention(F16),
    "float64 operands": lambda: attention(torch.float64),
    "int32 operands": lambda: attention(torch.int32),
    "bf16 lse": lambda: attention(lse=torch.zeros(2, 4, dtype=BF)),
    "float64 lse": lambda: attention(lse=torch.zeros(2, 4, dtype=torch.float64)),
    "transposed lse": lambda: attention(lse=torch.zeros(4, 2).T),
    "lse, every other row": lambda: attention(lse=torch.zeros(4, 4)[::2]),
    "offsets, every other one": lambda: attention(cu_q=torch.zeros(6).int()[::2]),
    "key offsets, every other one": lambda: attention(cu_k=torch.zeros(6).int()[::2]),
    "offsets of two dimensions": lambda: attention(cu_q=torch.zeros(3, 2).int(), cu_k=torch.zeros(3, 2).int()),
    "no offsets": lambda: attention(cu_q=torch.zeros(0).int(), cu_k=torch.zeros(0).int()),
}


@pytest.mark.parametrize("name", BAD_ATTENTION)
def test_attention_refuses(name):
    forward, backward, kw = BAD_ATTENTION[name]()
    with pytest.raises(ValueError):
        g.gpt2_op_attention_packed_forward(*forward, **kw)
    with pytest.raises(ValueError):
        g.gpt2_op_attention_packed_backward(*backward, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_refuses_tensors_that_are_not_on_the_device(dtype):
    for kw in (dict(), dict(status=torch.zeros(1).int()), dict(status=torch.zeros(1).long())):
        forward, backward, kw = attention(dtype, **kw)
        with pytest.raises(RuntimeError, match="current CUDA device"):
            g.gpt2_op_attention_packed_forward(*forward, **kw)
        with pytest.raises(RuntimeError, match="current CUDA device"):
            g.gpt2_op_attention_packed_backward(*backward, **kw)


def logprobs(**kw):
    n = 4
    c = dict(logp=torch.zeros(n), lse=torch.zeros(n), entropy=torch.zeros(n), logits=torch.zeros(n, 64, dtype=BF),
             targets=torch.zeros(n).int(), top_logp=torch.zeros(n, 3), top_ids=torch.zeros(n, 3).int(), status=None)
    c.update(kw)
    return [c[x] for x in ("logp", "lse", "entropy", "logits", "targets")] + [30], \
        {x: c[x] for x in ("top_logp", "top_ids", "status")}


BAD_LOGPROBS = {
    "float16 logits": dict(logits=torch.zeros(4, 64, dtype=F16)),
    "int64 targets": dict(targets=torch.zeros(4).long()),
    "few targets": dict(targets=torch.zeros(3).int()),
    "targets, every other one": dict(targets=torch.zeros(8).int()[::2]),
    "bf16 logp": dict(logp=torch.zeros(4, dtype=BF)),
    "float64 lse": dict(lse=torch.zeros(4, dtype=torch.float64)),
    "few lse": dict(lse=torch.zeros(2)),
    "lse of two dimensions": dict(lse=torch.zeros(4, 1)),
    "entropy, every other one": dict(entropy=torch.zeros(8)[::2]),
    "int64 ids": dict(top_ids=torch.zeros(4, 3).long()),
    "bf16 top": dict(top_logp=torch.zeros(4, 3, dtype=BF)),
    "few rows of alternatives": dict(top_logp=torch.zeros(2, 3), top_ids=torch.zeros(2, 3).int()),
    "transposed alternatives": dict(top_logp=torch.zeros(3, 4).T, top_ids=torch.zeros(3, 4).int().T),
    "alternatives of one dimension": dict(top_logp=torch.zeros(4), top_ids=torch.zeros(4).int()),
}


@pytest.mark.parametrize("name", BAD_LOGPROBS)
def test_logprobs_refuses(name):
    a, kw = logprobs(**BAD_LOGPROBS[name])
    with pytest.raises(ValueError):
        g.gpt2_op_token_logprobs(*a, **kw)


def logprobs_backward(**kw):
    n = 4
    c = dict(dlogits=torch.zeros(n, 64), logits=torch.zeros(n, 64), targets=torch.zeros(n).int(), lse=torch.zeros(n),
             entropy=torch.zeros(n), dlogp=torch.zeros(n), dlse=torch.zeros(n), dentropy=torch.zeros(n))
    c.update(kw)
    return [c[x] for x in ("dlogits", "logits", "targets", "lse", "entropy")] + [30], \
        {x: c[x] for x in ("dlogp", "dlse", "dentropy")}


@pytest.mark.parametrize("bad", [dict(dlogits=torch.zeros(4, 64, dtype=F16), logits=torch.zeros(4, 64, dtype=F16)),
                                 dict(targets=torch.zeros(4).long()), dict(targets=torch.zeros(3).int()),
                                 dict(lse=torch.zeros(4, dtype=BF)), dict(lse=torch.zeros(3)),
                                 dict(entropy=torch.zeros(8)[::2]), dict(dlogp=torch.zeros(4, dtype=BF)),
                                 dict(dlse=torch.zeros(4).double()), dict(dentropy=torch.zeros(2))],
                         ids=lambda b: ",".join(f"{k} {tuple(v.shape)} {v.dtype}" for k, v in b.items()))
def test_logprobs_backward_refuses(bad):
    a, kw = logprobs_backward(**bad)
    with pytest.raises(ValueError):
        g.gpt2_op_token_logprobs_backward(*a, **kw)


def test_logprobs_refuses_tensors_that_are_not_on_the_device():
    a, kw = logprobs()
    with pytest.raises(RuntimeError, match="current CUDA device"):
        g.gpt2_op_token_logprobs(*a, **kw)
    a, kw = logprobs_backward()
    with pytest.raises(RuntimeError, match="current CUDA device"):
        g.gpt2_op_token_logprobs_backward(*a, **kw)
