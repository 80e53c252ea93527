"""Pins of the expert-block oracle (RMS norm, routing, expert layer of a few tokens)
against things other than itself: torch's autograd in float64, central differences,
library sorts, closed forms and the grouped-MLP oracle."""
import numpy as np
import pytest
import torch

import oracle
from oracle import expert_block as eb


def t64(a):
    return torch.from_numpy(np.asarray(a, np.float64)).requires_grad_(True)


@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm_and_backward_match_autograd(with_residual):
    rng = np.random.default_rng(1)
    x, r, g = rng.normal(0, 2, (7, 24)), rng.normal(0, 1, (7, 24)), rng.normal(1, 0.3, 24)
    dy, dh = rng.normal(0, 1, (7, 24)), rng.normal(0, 1, (7, 24))
    X, R, G = t64(x), t64(r), t64(g)
    H = X + R if with_residual else X * 1.0
    Y = torch.nn.functional.rms_norm(H, (24,), G, 1e-5)
    h, y = eb.rmsnorm(x, g, 1e-5, r if with_residual else None)
    assert np.allclose(h, H.detach().numpy(), rtol=1e-15) and np.allclose(y, Y.detach().numpy(), rtol=1e-13)
    ((Y * torch.from_numpy(dy)).sum() + (H * torch.from_numpy(dh)).sum()).backward()
    dx, dg = eb.rmsnorm_backward(dy, h, g, 1e-5, dh)
    assert np.allclose(dx, X.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(dg, G.grad.numpy(), rtol=1e-12, atol=1e-13)


def test_rmsnorm_closed_forms():
    h, y = eb.rmsnorm(np.array([[3.0, -3.0, 3.0, 3.0], [0.0] * 4]), np.array([1.0, 2.0, 0.0, -1.0]), 0.0)
    assert y[0].tolist() == [1.0, -2.0, 0.0, -1.0]
    assert np.isnan(y[1]).all()
    assert (eb.rmsnorm(np.zeros((1, 4)), np.ones(4), 1e-6)[1] == 0).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_matches_torch_and_backward_matches_autograd(sigmoid, renormalize):
    rng = np.random.default_rng(2)
    l, dw, k = rng.normal(0, 2, (11, 9)), rng.normal(0, 1, (11, 4)), 4
    ids, w = eb.route(l, k, sigmoid, renormalize)
    L = t64(l)
    S = torch.sigmoid(L) if sigmoid else torch.softmax(L, 1)
    top, at = torch.topk(S, k, dim=1)
    W = top / top.sum(1, keepdim=True) if renormalize else top
    assert np.array_equal(ids, at.numpy()) and np.allclose(w, W.detach().numpy(), rtol=1e-13)
    (W * torch.from_numpy(dw)).sum().backward()
    d = eb.route_backward(l, ids, dw, sigmoid, renormalize)
    assert np.allclose(d, L.grad.numpy(), rtol=1e-11, atol=1e-14)
    # central differences with the choice held fixed (the step leaves the order as it is)
    step, gaps = 1e-6, np.diff(np.sort(l, axis=1), axis=1).min()
    assert gaps > 4 * step
    for t, e in ((0, int(ids[0, 0])), (3, int(ids[3, 3])), (5, 0)):
        up, down = l.copy(), l.copy()
        up[t, e] += step
        down[t, e] -= step
        diff = (eb.route(up, k, sigmoid, renormalize)[1] - eb.route(down, k, sigmoid, renormalize)[1]) / (2 * step)
        assert abs((diff * dw).sum() - d[t, e]) < 1e-8


def test_route_masks_and_ties():
    inf = np.inf
    l = np.array([[1.0, 1.0, 1.0, 1.0], [-inf, 2.0, -inf, -inf], [-inf] * 4, [np.nan, 0.0, inf, inf], [0.0, -0.0, 0.0, -1.0]])
    ids, w = eb.route(l, 2)
    assert ids.tolist() == [[0, 1], [1, 0], [0, 1], [2, 3], [0, 1]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [0.5, 0.5], [0.5, 0.5]]
    d = eb.route_backward(l, ids, np.ones((5, 2)), sigmoid=True, renormalize=False)
    assert d[2].tolist() == [0.0] * 4 and d[1, 0] == 0.0


def test_plan_is_the_stable_order():
    rng = np.random.default_rng(3)
    ids = np.stack([rng.permutation(6)[:3] for _ in range(20)])
    splits, rows, slots = eb.plan(ids, 6)
    order = np.argsort(ids.reshape(-1), kind="stable")
    assert np.array_equal(slots, order) and np.array_equal(rows.reshape(-1)[order], np.arange(60))
    assert np.array_equal(splits, np.bincount(ids.reshape(-1), minlength=6))


def test_moe_is_the_grouped_mlp_over_the_plan():
    rng = np.random.default_rng(4)
    T, E, k, K, F, N = 6, 5, 2, 16, 8, 24
    x, res = rng.normal(0, 1, (T, K)), rng.normal(0, 1, (T, N))
    w1, w2 = rng.normal(0, 0.3, (E, 2 * F, K)), rng.normal(0, 0.3, (E, N, F))
    b1, b2 = rng.normal(0, 0.3, (E, 2 * F)), rng.normal(0, 0.3, (E, N))
    ids, w = eb.route(rng.normal(0, 1, (T, E)), k)
    splits, rows, slots = eb.plan(ids, E)
    _, _, z = oracle.mlp_forward(x[slots // k], w1, b1, w2, b2, splits, "f64")
    y = res + (z[rows] * w[..., None]).sum(1)
    assert np.allclose(eb.moe(x, ids, w, w1, w2, b1, b2, res), y, rtol=1e-12, atol=1e-13)
    gone = ids.copy()
    gone[2] = [-1, E]
    assert np.array_equal(eb.moe(x, gone, w, w1, w2, b1, b2, res)[2], res[2])
