"""Token routing at logits far from zero, against the float64 oracle.

With e = 2^-24, a score s = sigmoid(l) of fp32 operations has a relative error of (|l| + 6) e
(the exponential's argument is exact, its result within 2 e; |l| e covers a product in it), its
slope 1 - s = sigmoid(-l) the same, a sum over k positive terms k e more: a product of two
scores and a slope, divided by such a sum, is within n = (4 max|l| + k + 40) e of its own size,
and a difference dw - sum(dw w) within n of its terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import to64
from oracle import expert_block as eb
from test_gpu_route import BF16, F16, F32, FLOOR, SCORE, U, E24, forward

pytestmark = pytest.mark.gpu
DEV = "cuda"


def backward(l, ids, dw, sigmoid, renorm):
    out = torch.full(l.shape, float("nan"), dtype=l.dtype, device=DEV)
    gl.gl_route_backward(l.to(DEV), torch.from_numpy(ids).int().to(DEV), dw.to(DEV), out, score=SCORE[sigmoid], renormalize=renorm)
    return to64(out)


def away_from_zero(seed, T, E, dtype, lo, hi):
    """Logits of either sign with magnitudes lo ... hi."""
    g = torch.Generator().manual_seed(seed)
    size = lo + (hi - lo) * torch.rand(T, E, generator=g)
    return (size * (torch.randint(0, 2, (T, E), generator=g) * 2 - 1)).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("lo,hi", [(0, 8), (8, 18), (17, 40), (40, 80)])
def test_sigmoid_gradient_keeps_its_relative_precision(dtype, renorm, lo, hi):
    T, E, k = 130, 24, 5
    l = away_from_zero(lo, T, E, dtype, lo, hi)
    L, dw = to64(l), torch.randn(T, k, generator=torch.Generator().manual_seed(hi))
    ids, w = eb.route(L, k, True, renorm)
    got, ref = backward(l, ids, dw, True, renorm), eb.route_backward(L, ids, dw.numpy(), True, renorm)
    c, D = np.take_along_axis(L, ids, 1), dw.numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        slope = 1 / (1 + np.exp(c))  # 1 - s without its cancellation
    mean = (D * w).sum(1, keepdims=True) if renorm else 0.0
    exact, mag = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(exact, ids, slope * w * (D - mean), 1)
    np.put_along_axis(mag, ids, slope * w * (np.abs(D) + ((np.abs(D) * w).sum(1, keepdims=True) if renorm else 0.0)), 1)
    assert np.allclose(ref, exact, rtol=1e-6, atol=1e-14)  # the oracle's 1 - s, in 64 bits, as far as it goes
    lim = U[dtype] * np.abs(exact) + (4 * hi + k + 40) * E24 * mag + FLOOR[dtype]
    bad = ~(np.abs(got - exact) <= lim)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size}, worst {np.max(np.abs(got - exact) / (lim + 1e-300)):.3g} times"


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("E,k", [(24, 5), (300, 8), (3, 3)])
def test_renormalised_sigmoids_below_the_range_of_fp32(dtype, E, k):
    """Every logit so low that fp32 holds its sigmoid as 0 or subnormally: the weights are
    still the scores divided by their sum, and the gradient theirs."""
    T = 40
    l = (-torch.linspace(80, 700, T)[:, None] - 6 * torch.rand(T, E, generator=torch.Generator().manual_seed(E))).to(dtype)
    L, dw = to64(l), torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    got = forward(l.to(DEV), k, True, True)
    ids, w = eb.route(L, k, True, True)
    assert np.array_equal(got["ids"].cpu().numpy(), ids)
    n = (4 * 20 + k + 40) * E24  # the exponentials' arguments are differences of at most 6 and a step of the type
    assert (np.abs(to64(got["weights"]) - w) <= n * w).all()
    D = dw.numpy().astype(np.float64)
    exact, mag = np.zeros((T, E)), np.zeros((T, E))  # slopes are 1
    np.put_along_axis(exact, ids, w * (D - (D * w).sum(1, keepdims=True)), 1)
    np.put_along_axis(mag, ids, w * (np.abs(D) + (np.abs(D) * w).sum(1, keepdims=True)), 1)
    assert (np.abs(backward(l, ids, dw, True, True) - exact) <= U[dtype] * np.abs(exact) + n * mag + FLOOR[dtype]).all()
    alone = forward(l.to(DEV), k, True, False)["weights"]  # not renormalised: the small numbers themselves
    s = np.exp(np.take_along_axis(L, ids, 1))
    assert (np.abs(to64(alone) - s) <= (4 * 90 + 40) * E24 * s + 2.0 ** -148).all()


def test_a_types_lowest_value_masks_sigmoids():
    for dtype in (F32, BF16):
        l = torch.full((3, 9), float(torch.finfo(dtype).min), dtype=dtype)
        l[1, 4] = -1.0
        l[2, 2] = l[2, 7] = -800.0
        got = forward(l.to(DEV), 2, True, True)
        assert got["ids"].tolist() == [[0, 1], [4, 0], [2, 7]] and got["weights"].tolist() == [[0, 0], [1, 0], [0, 0]]


@pytest.mark.parametrize("E,k", [(12, 4), (300, 6)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_slots_take_no_part_in_the_gradient(E, k, bad):
    """dweights of slots that a mask left (weight 0) may be NaN or infinite."""
    g = torch.Generator().manual_seed(E)
    l = torch.randn(9, E, generator=g)
    l[1:, 2:] = -float("inf")  # two experts left
    l[8] = float("nan")  # none
    dw = torch.randn(9, k, generator=g)
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids, w = eb.route(to64(l), k, sigmoid, renorm)
            broken = torch.where(torch.from_numpy(w) == 0, torch.tensor(bad), dw)
            got = backward(l, ids, broken, sigmoid, renorm)
            assert np.array_equal(got, backward(l, ids, dw, sigmoid, renorm))
            assert np.abs(got[1:, 2:]).max() == 0 and np.abs(got[8]).max() == 0
