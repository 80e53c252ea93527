"""Scales of the 8-bit integer products over fp32's whole range: y = sum x_scale w_scale + b is finite
where the formula is, 0 where the sum is 0, and infinite where the formula passes the type.

Tolerance: a sum is exact below 2^24, three roundings of 2^-24 relative (two scales and the bias),
half of the smallest subnormal, and the output's own rounding."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import to64
from oracle import gated
from test_gpu_glu import check, glu_limits, half_step

pytestmark = pytest.mark.gpu
DEV, F32, BF, K = "cuda", torch.float32, torch.bfloat16, 128
# with each other: products of 1e-42 .. 1e76, and ordinary results from scales far apart
SCALES = [1.0, 1e-12, 1e-30, -1e-38, 1e-44, 1e20, -1e25, 1e30, 3e38, 0.0, 2.0 ** 96, 2.0 ** 97, 2.0 ** -126]
SUMS = [0, 1, -127, 127 * 127, 100 * 127 * 127]


def problem(T, N, K, bias, out):
    """Row t has scale t, column n scale n / 5 and the sum n % 5: x is 127 at a hundred places of K and 1
    at the next, and w picks from them."""
    x, w = torch.zeros(T, K, dtype=torch.int8), torch.zeros(1, N, K, dtype=torch.int8)
    x[:, :100] = 127
    w[0, 1::5, 100] = 1
    w[0, 2::5, 0] = -1
    w[0, 3::5, 0] = 127
    w[0, 4::5, :100] = 127
    x[:, 100] = 1
    xs = torch.tensor([SCALES[t % len(SCALES)] for t in range(T)], dtype=F32)
    ws = torch.tensor([SCALES[(n // 5) % len(SCALES)] for n in range(N)], dtype=F32)[None]
    b = torch.linspace(-2, 2, N).to(out)[None] if bias else None
    space = gl.new_workspace(1)
    gl.gl_offsets(torch.tensor([T], dtype=torch.int64, device=DEV), T, space)
    host = (x, xs, w, ws, b)
    return host, [None if t is None else t.to(DEV) for t in host], space


def reference(host):
    x, xs, w, ws, b = (None if t is None else to64(t) for t in host)
    s = gated.product(x, w, None, [x.shape[0]])
    h = s * xs[:, None] * ws
    assert set(np.unique(s)) == set(SUMS)
    return h + (0.0 if b is None else b), 3 * 2.0 ** -24 * (np.abs(h) + (0.0 if b is None else np.abs(b))) + 2.0 ** -150


# kernel: rows and weight rows
SIZES = {"32x64 parts": (13, 72), "32x64": (13, 16384), "128x128": (26, 16384), "256 ragged": (200, 24000),
         "256 full": (1030, 9000)}


@pytest.mark.parametrize("kernel", SIZES)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("out", [F32, BF])
def test_product(kernel, bias, out):
    T, N = SIZES[kernel]
    host, (x, xs, w, ws, b), space = problem(T, N, K, bias, out)
    y = torch.empty(T, N, dtype=out, device=DEV)
    gl.gl_forward_int8(x, xs, w, ws, y, space, bias=b)
    ref, e = reference(host)
    got = to64(y)
    lim = e + half_step(out, ref)
    top = torch.finfo(out).max
    over = np.abs(ref) - lim > top * (1 + torch.finfo(out).eps / 4)
    near = (np.abs(ref) + lim > top) & ~over
    assert not near.any()
    assert over.any() and (got[over] == np.sign(ref[over]) * np.inf).all()
    check(torch.from_numpy(np.where(over, 0.0, got)), np.where(over, 0.0, ref), lim, "y")


@pytest.mark.parametrize("T,F", [(13, 40), (1030, 4104)])
def test_gated_product(T, F):
    """Gates whose sums are 0 under scales whose product overflows: what is left is the bias."""
    g = torch.Generator().manual_seed(F)
    x, w = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8) for s in ((T, K), (1, 2 * F, K)))
    w[0, :F] = 0
    xs, ws, b = torch.full((T,), 1e25), torch.full((1, 2 * F), 1e20), torch.randn(1, 2 * F, generator=g)
    ws[0, F:] = 1e-28
    space = gl.new_workspace(1)
    gl.gl_offsets(torch.tensor([T], dtype=torch.int64, device=DEV), T, space)
    a = torch.empty(T, F, dtype=F32, device=DEV)
    gl.gl_glu_forward_int8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), a, space, bias=b.to(DEV))
    v = [to64(t) for t in (x, xs, w, ws, b)]
    h, mag = gated.product_int8(*v, [T]), np.abs(gated.product_int8(*v[:4], None, [T]))
    check(a, *glu_limits("silu", h, 3 * 2.0 ** -24 * (mag + np.abs(v[4])), F32), "a")
