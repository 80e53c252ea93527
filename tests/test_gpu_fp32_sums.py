"""Long contractions of the fp32 gated layer on its small tiles: sums go in chunks of 256 values, whose
sums are added up.

Of n products in that order a sum is off by at most (256 + n / 256 + 2) 2^-24 of the sum of their
magnitudes.  The inputs make a single chain fail that: one product of 1, the others 2^-27, which
are each lost against 1 (n 2^-27, 6e-5 at 2^13, where 1.8e-5 is allowed), but not their chunks' sums."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def limit(n):
    return (256 + n / 256 + 2) * 2.0 ** -24


def workspace(T):
    ws = gl.new_workspace(1)
    gl.gl_offsets(torch.tensor([T], dtype=torch.int64, device=DEV), T, ws)
    return ws


def new(*s):
    return torch.empty(*s, device=DEV)


# kernel: T, K, F
FORWARD = {"few": (8, 1 << 15, 64), "32x64 parts": (40, 1 << 14, 64), "32x64": (100, 1 << 14, 4096),
           "64x64": (300, 1 << 14, 4096)}
DX = {"32x64 parts": (40, 64, 1 << 13), "32x64": (100, 6400, 1 << 13), "64x64": (300, 5760, 1 << 13)}


@pytest.mark.parametrize("kernel", FORWARD)
def test_forward(kernel):
    T, K, F = FORWARD[kernel]
    x, w, h = torch.full((T, K), 2.0 ** -14, device=DEV), torch.full((1, 2 * F, K), 2.0 ** -13, device=DEV), new(T, 2 * F)
    x[:, 0], w[:, :, 0] = 1, 1
    gl.gl_glu_forward(x, w, new(T, F), workspace(T), h=h)
    ref = 1 + (K - 1) * 2.0 ** -27
    off = float((h.double() / ref - 1).abs().max())
    assert off <= limit(K), off


@pytest.mark.parametrize("kernel", DX)
def test_dx(kernel):
    T, K, F = DX[kernel]
    h = torch.full((T, 2 * F), 2.0 ** -13, device=DEV)  # the other half; dh of the gate's half is it times 1
    h[:, :F], h[:, F] = 30, 1  # SiLU's slope at 30 is 1
    w = torch.zeros(1, 2 * F, K, device=DEV)
    w[:, :F] = 2.0 ** -14
    w[:, 0] = 1
    dh, dx, dw = new(T, 2 * F), new(T, K), new(1, 2 * F, K)
    gl.gl_glu_backward(torch.zeros(T, K, device=DEV), w, torch.ones(T, F, device=DEV), dh, dx, dw, workspace(T), h=h)
    assert bool((dh[:, 0] == 1).all()) and bool((dh[:, 1:F] == 2.0 ** -13).all())
    ref = 1 + (F - 1) * 2.0 ** -27
    off = float((dx.double() / ref - 1).abs().max())
    assert off <= limit(2 * F), off


@pytest.mark.parametrize("accumulate", [False, True])
def test_dw(accumulate):
    """dW, whose contraction is the rows of a group."""
    T, K, F = 1 << 14, 72, 40
    h = torch.full((T, 2 * F), 2.0 ** -13, device=DEV)
    h[:, :F], h[0, F:] = 30, 1
    x = torch.full((T, K), 2.0 ** -14, device=DEV)
    x[0] = 1
    dh, dw = new(T, 2 * F), torch.ones(1, 2 * F, K, device=DEV)
    gl.gl_glu_backward(x, torch.zeros(1, 2 * F, K, device=DEV), torch.ones(T, F, device=DEV), dh, None, dw, workspace(T),
                       h=h, accumulate=accumulate)
    ref = 1 + (T - 1) * 2.0 ** -27
    got = dw[0, :F].double() - (1.0 if accumulate else 0.0)
    off = float((got / ref - 1).abs().max())
    assert off <= limit(T) + (2.0 ** -23 if accumulate else 0.0), off


def test_sums_of_ordinary_values_are_nearer_than_one_chain_of_them():
    """5 groups, 221 rows, K 7040, 2F 12080: one chain is off by 2.0e-6 of the norm (measured), random roundings of
    256 values and then of 48 sums by sqrt(256 / 12080) and sqrt(48 / 12080) of that, 2.9e-7 and 1.3e-7; twice
    what both make together."""
    m, K, F = [44, 45, 44, 44, 44], 7040, 6040
    T = sum(m)
    g = torch.Generator(DEV).manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    w, dh, dx, dw = r(5, 2 * F, K).mul_(K ** -0.5), new(T, 2 * F), new(T, K), new(5, 2 * F, K)
    ws = gl.new_workspace(5)
    gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), T, ws)
    gl.gl_glu_backward(r(T, K), w, r(T, F), dh, dx, dw, ws, h=r(T, 2 * F))
    ends = np.cumsum(m)
    ref = torch.cat([dh[e - n:e].double() @ w[i].double() for i, (n, e) in enumerate(zip(m, ends))])
    off = float((dx.double() - ref).norm() / ref.norm())
    assert off < 6.4e-7, off
