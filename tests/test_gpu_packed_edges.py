"""Calls at the edges of what packed attention and the token log-probabilities allow, against the float64 oracle."""
import numpy as np
import pytest

from oracle import packed_ref as P
from step_gpt_train_gb300 import data
from tests._gpu_util import dev, host, inputs
from tests.test_gpu_packed import Packed, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    from step_gpt_train_gb300 import gpt2 as g
    g.load_library(build=True)
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lq,hidden", [(300, 128), (200, 130), (200, 256), (1, 200)])
def test_attention_first_keys_score_minus_infinity(torch_cuda, lq, hidden, mode):
    """A query whose first keys all score -inf (products past fp32's range) is the query without them."""
    torch = torch_cuda
    lk = hidden + max(lq, 90)
    c = Packed(torch, 41, [lq], [lk], 4, 2, 64, mode, before=0, after=0)
    first = slice(0, hidden)
    c.q[..., 0] = float(data.round_to_bf16(np.float32([1e20]))[0])
    c.k[..., 0] = 0.0
    c.k[first, :, 0] = -c.q[0, 0, 0]
    c.tq.copy_(dev(c.q.astype(np.float32), mode))
    c.tk.copy_(dev(c.k.astype(np.float32), mode))
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    rest = slice(hidden, lk)
    cu_k = np.array([0, lk - hidden])
    o, lse, bo, bl = P.attention_forward(c.q, c.k[rest], c.v[rest], c.cu_q, cu_k, mode)
    within(host(c.o), o, bo, "o")
    within(host(c.lse), lse, bl, "lse")
    dq, dk, dv, bq, bk, bv = P.attention_backward(c.dout, c.q, c.k[rest], c.v[rest], c.cu_q, cu_k, mode)
    within(host(c.dq), dq, bq, "dq")
    within(host(c.dk)[rest], dk, bk, "dk")
    within(host(c.dv)[rest], dv, bv, "dv")
    assert not c.dk[first].any() and not c.dv[first].any()


@pytest.mark.parametrize("mode", [1, 0], ids=["bf16", "fp32"])
def test_attention_runs_of_items_without_keys(torch_cuda, mode):
    """Many work items in a row that meet no key (longer than a processor's share of them), among some that do."""
    r = np.random.default_rng(5)
    lq = [int(x) for x in r.integers(1, 300, 900)]
    lk = [0] * len(lq)
    lk[100], lk[101], lk[500], lq[700], lk[700] = 200, 7, 40, 2000, 300
    c = Packed(torch_cuda, 47, lq, lk, 4, 2, 64, mode)
    c.forward()
    c.backward()
    c.check()
