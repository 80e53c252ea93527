"""The mixture-of-experts block of examples/expert_block.py: its two forward paths against
the float64 oracle and each other, and its gradients against autograd in float64.

Bounds: every intermediate of the 16-bit path (n, logits, h, a, z and their gradients) is
rounded to bf16, half an ulp of 2^-8 relative each.  Such errors enter an output as a sum of
about independent terms, so an output of r roundings in a chain is held to 2 r 2^-8 of its
norm: the forward has 4 (n, h, a, z), the gradients at most 8.  In fp32 the same chains are
held to 1e-4, far above their roundings, far below a wrong term.  The choice of experts is
taken from the path itself: a near tie may fall either way between two precisions.
"""
import os
import sys

import numpy as np
import pytest
import torch

from gl_testutil import to64
from oracle import expert_block as eb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from expert_block import ExpertBlock  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORWARD = {torch.bfloat16: 8 * 2.0 ** -8, torch.float32: 1e-4}
BACKWARD = {torch.bfloat16: 16 * 2.0 ** -8, torch.float32: 1e-4}


def off(got, ref):
    return float(np.linalg.norm(to64(got) - ref) / np.linalg.norm(ref))


def make(T, dtype):
    block = ExpertBlock(features=128, ffn=64, experts=16, top_k=3, dtype=dtype, seed=T)
    g = torch.Generator().manual_seed(T)
    x, res, dy = ((torch.randn(T, 128, generator=g)).to(dtype).to(DEV) for _ in range(3))
    return block, x, res, dy


@pytest.mark.parametrize("T", [1, 7, 40, 64, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward_paths(T, dtype):
    block, x, res, _ = make(T, dtype)
    y, c = block.forward(x, res)
    s, n = eb.rmsnorm(to64(x), to64(block.gamma), block.eps, to64(res))
    logits = n @ to64(block.wr)[0].T
    ids = c["ids"].cpu().numpy()
    w = np.take_along_axis(logits, ids.astype(np.int64), 1)
    w = np.exp(w - w.max(1, keepdims=True))
    ref = eb.moe(n, ids, w / w.sum(1, keepdims=True), to64(block.w1), to64(block.w2), residual=s)
    assert off(y, ref) < FORWARD[dtype]
    if T <= 64:
        d = block.decode(x, res)
        assert off(d, ref) < FORWARD[dtype]


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_against_autograd(T, dtype):
    block, x, res, dy = make(T, dtype)
    y, c = block.forward(x, res)
    got = block.backward(dy, c)
    p = {n: getattr(block, n).double().cpu().requires_grad_(True) for n in ("gamma", "wr", "w1", "w2")}
    X = x.double().cpu().requires_grad_(True)
    s = X + res.double().cpu()
    n = torch.nn.functional.rms_norm(s, (128,), p["gamma"], block.eps)
    ids = c["ids"].long().cpu()
    w = torch.softmax((n @ p["wr"][0].T).gather(1, ids), 1)
    out = s.clone()
    for j in range(ids.shape[1]):
        h = torch.einsum("tk,tfk->tf", n, p["w1"][ids[:, j]])
        a = torch.nn.functional.silu(h[:, :64]) * h[:, 64:]
        out = out + w[:, j:j + 1] * torch.einsum("tf,tnf->tn", a, p["w2"][ids[:, j]])
    (out * dy.double().cpu()).sum().backward()
    assert off(y, out.detach().numpy()) < FORWARD[dtype]
    for name, ref in (("x", X.grad), ("gamma", p["gamma"].grad), ("wr", p["wr"].grad), ("w1", p["w1"].grad), ("w2", p["w2"].grad)):
        assert off(got[name], ref.numpy()) < BACKWARD[dtype], name
