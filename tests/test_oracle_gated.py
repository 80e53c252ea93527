"""The oracle of the gated layer and of the 8-bit integer product against torch's own functions,
autograd in float64 and hand-worked values."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import gated

TORCH = {"silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}


@pytest.mark.parametrize("name", gated.ACTS)
def test_activation_and_slope(name):
    v = torch.linspace(-12, 12, 4801, dtype=torch.float64, requires_grad=True)
    y = TORCH[name](v)
    (d,) = torch.autograd.grad(y.sum(), v)
    np.testing.assert_allclose(gated.act(name, v.detach().numpy()), y.detach().numpy(), rtol=1e-9, atol=1e-15)
    np.testing.assert_allclose(gated.slope(name, v.detach().numpy()), d.numpy(), rtol=1e-9, atol=1e-14)


@pytest.mark.parametrize("name", gated.ACTS)
def test_layer_and_gradient_against_autograd(name):
    g = torch.Generator().manual_seed(3)
    m, K, Fo = [3, 0, 5], 6, 4
    x = torch.randn(8, K, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(3, 2 * Fo, K, generator=g, dtype=torch.float64, requires_grad=True)
    b = torch.randn(3, 2 * Fo, generator=g, dtype=torch.float64, requires_grad=True)
    da = torch.randn(8, Fo, generator=g, dtype=torch.float64)
    h = torch.cat([x[r] @ w[i].t() + b[i] for i, r in gated.groups(m)])
    a = TORCH[name](h[:, :Fo]) * h[:, Fo:]
    dx, dw, db = torch.autograd.grad((a * da).sum(), (x, w, b))
    xn, wn, bn = (t.detach().numpy() for t in (x, w, b))
    hn = gated.product(xn, wn, bn, m)
    np.testing.assert_allclose(gated.glu(name, hn), a.detach().numpy(), rtol=1e-12)
    got = gated.glu_backward(xn, wn, gated.glu_grad(name, hn, da.numpy()), m)
    for o, t in zip(got, (dx, dw, db)):
        np.testing.assert_allclose(o, t.numpy(), rtol=1e-10, atol=1e-12)


def test_quantize_int8_hand_worked():
    q, s = gated.quantize_int8(np.array([[127.0, 0.5, 1.5, -2.5], [0, 0, 0, 0], [-2.0, 1.0, 0.25, 0]]))
    assert q.tolist() == [[127, 0, 2, -2], [0, 0, 0, 0], [-127, 64, 16, 0]]  # 63.5 and 15.875; ties to even
    assert s[0] == 1.0 and s[1] == np.float32(np.float32(2.0 ** -100) / np.float32(127)) and s[2] == np.float32(2 / 127)
    q, s = gated.quantize_int8(np.array([[np.inf, 1.0], [np.nan, 1.0], [1.0, 1.0]]))
    assert q.tolist() == [[0, 0], [0, 0], [127, 127]] and np.isnan(s[:2]).all() and np.isfinite(s[2])


def test_product_int8_is_the_dequantized_product():
    g = np.random.default_rng(5)
    x, w = g.integers(-128, 128, (7, 32)), g.integers(-128, 128, (2, 6, 32))
    xs, ws, b = g.random(7), g.random((2, 6)), g.standard_normal((2, 6))
    m = [4, 3]
    ref = gated.product(x * xs[:, None], w * ws[..., None], b, m)
    np.testing.assert_allclose(gated.product_int8(x, xs, w, ws, b, m), ref, rtol=1e-12, atol=1e-12)
