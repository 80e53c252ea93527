"""GELU's negative tail in the gated layer: v Phi(v) and its slope relative to their own size, for gates
from -9 to -3, where Phi is 1e-19 to 1e-3.

Tolerances, with t = 2^-23.  If Phi comes from erfc: its argument is v times a constant, both rounded, so
off by t relative, Phi's relative change is at most v^2 + 1 times that (the normal density over Phi
is at most |v| + 1 / |v|), and erfc itself is within 16 t.  If it comes from exp(-v^2 / 2) times a
polynomial of 1 / (1 + c |v|): the exponent is off by at most 3 roundings, 0.75 v^2 t, exp2, the
reciprocal and the polynomial by 6 t.  The density likewise.  Two or three products by exact
values follow.  Either way at most (v^2 + 21) t of Phi + |v| density, and the output's own rounding."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import to64
from oracle import gated
from test_gpu_glu import TYPES, check, half_step

pytestmark = pytest.mark.gpu
DEV, K = "cuda", 64
SIZES = [(1, 64), (70, 520), (1000, 4096)]  # in 16 bits the contraction in two parts, twice, and tiles of 256


def gates(F, dtype):
    return torch.linspace(-9, -3, F).to(dtype)


def tail(v):
    """(act, slope, their allowed arithmetic error) in float64 for gates v."""
    phi = gated.act("gelu", v) / v
    density = phi - gated.slope("gelu", v)  # |v| times it
    step = (v * v + 21) * 2.0 ** -23
    return gated.act("gelu", v), gated.slope("gelu", v), step * np.abs(v) * phi, step * (phi + density)


def workspace(T):
    ws = gl.new_workspace(1)
    gl.gl_offsets(torch.tensor([T], dtype=torch.int64, device=DEV), T, ws)
    return ws


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,F", SIZES)
def test_forward(T, F, dtype):
    """No tokens' part: the gate is the bias, the other half 1."""
    v = gates(F, dtype)
    b = torch.cat([v, torch.ones(F, dtype=dtype)])[None].to(DEV)
    x, w = torch.zeros(T, K, dtype=dtype, device=DEV), torch.ones(1, 2 * F, K, dtype=dtype, device=DEV)
    a = torch.empty(T, F, dtype=dtype, device=DEV)
    gl.gl_glu_forward(x, w, a, workspace(T), bias=b, act=gl.GL_GLU_GELU)
    act, _, e, _ = tail(to64(v))
    ref = np.broadcast_to(act, (T, F))
    check(a, ref, e + half_step(dtype, ref), "a")


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,F", SIZES)
def test_backward(T, F, dtype, kept):
    v = gates(F, dtype)
    b = torch.cat([v, torch.ones(F, dtype=dtype)])[None].to(DEV)
    x, w = torch.zeros(T, K, dtype=dtype, device=DEV), torch.ones(1, 2 * F, K, dtype=dtype, device=DEV)
    new = lambda *s: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    a, dh, dw = new(T, F), new(T, 2 * F), new(1, 2 * F, K)
    da = torch.ones(T, F, dtype=dtype, device=DEV)
    gl.gl_glu_backward(x, w, da, dh, None, dw, workspace(T), h=b.expand(T, 2 * F).contiguous() if kept else None,
                       bias=b, a=a, act=gl.GL_GLU_GELU)
    act, slope, e, es = (np.broadcast_to(t, (T, F)) for t in tail(to64(v)))
    check(a, act, e + half_step(dtype, act), "a")
    check(dh[:, :F], slope, es + half_step(dtype, slope), "dh of the gate")
    check(dh[:, F:], act, e + half_step(dtype, act), "dh of the other half")
