"""The gated layer's small tiles and their choice, and the backward's products whose operands or
outputs pass the last-level cache (tolerances as in test_gpu_glu.py)."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import nan_tail, to64
from oracle import gated
from test_gpu_glu import ACTS, Layer, V, check, glu_limits, grad_limits, half_step
from test_gpu_int8 import Int8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# (type, rows of the groups, K, F): rows by weight rows of the forward's tiles
FORWARD = {
    "32x32": (BF, [33, 0, 1, 40], 264, 136),
    "32x32 few rows": (F16, [7, 0, 17, 1] * 4, 200, 1048),     # 6 rows a group, 594 tiles of 64
    "64x64": (BF, [20, 0, 70, 30] * 2, 264, 776),              # 275 tiles of 64
    "64x64 f16": (F16, [20, 0, 65, 5, 0, 0, 129], 72, 840),
    "32x64 f32": (F32, [33, 0, 1, 40], 100, 136),
    "64x64 f32": (F32, [300, 2, 513], 132, 1000),              # 928 tiles of 32
    "contraction split f32": (F32, [3, 0, 9, 4], 1028, 1020),
}


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("path", FORWARD)
def test_forward_tiles(path, name):
    dtype, m, K, F = FORWARD[path]
    L = Layer(m, K, F, dtype, seed=K)
    a, h = nan_tail(L.T + 2, F, L.T, dtype, DEV), L.new(L.T, 2 * F)
    gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h, act=ACTS[name])
    ref_h, e = L.h()
    check(a[:L.T], *glu_limits(name, ref_h, e, dtype), "a")
    check(h, ref_h, e + half_step(dtype, ref_h), "h")
    assert torch.isnan(a[L.T:]).all()
    dh, dw, a2 = L.new(L.T, 2 * F), L.new(L.G, 2 * F, K), L.new(L.T, F)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, None, dw, L.ws, bias=L.db_, a=a2, act=ACTS[name])
    check(dh, *grad_limits(name, ref_h, e, to64(L.da), dtype), "dh")
    check(a2, *glu_limits(name, ref_h, e, dtype), "a again")


@pytest.mark.parametrize("gate", [None, *ACTS])
@pytest.mark.parametrize("m,K,N", [([33, 0, 1, 40], 272, 144), ([15, 0, 17, 1] * 8, 144, 1056), ([600, 40], 400, 272)],
                         ids=str)
def test_int8_tiles(m, K, N, gate):
    """Tiles of 32 rows by 64: 19 rows a group, 8 rows, 320 rows."""
    P = Int8(m, K, N, BF, seed=K)
    h, e = P.h()
    y = nan_tail(P.T + 2, N // 2 if gate else N, P.T, BF, DEV)
    if gate:
        gl.gl_glu_forward_int8(*P.args, y, P.ws, bias=P.bias, act=ACTS[gate])
        check(y[:P.T], *glu_limits(gate, h, e, BF), "a")
    else:
        gl.gl_forward_int8(*P.args, y, P.ws, bias=P.bias)
        check(y[:P.T], h, e + half_step(BF, h), "y")
    assert torch.isnan(y[P.T:]).all()


# (type, rows of the groups, K, F)
BACKWARD = {
    "dx 32x64": (BF, [33, 0, 1, 70], 264, 72),
    "dx 64": (F16, [100, 0, 300, 257], 1032, 104),             # 425 tiles of 32
    "dx 32x64 f32": (F32, [33, 0, 1, 70], 260, 36),
    "dx 64 f32": (F32, [300, 2, 513], 2052, 68),               # 957 tiles of 32
    "dx 256, dW stored once": (BF, [100, 0, 140, 500, 1, 59, 0, 8], 4104, 2056),  # 270 MB of weights
    "dx 32x64, once f32": (F32, [2, 0, 7, 33, 1, 9, 0, 8], 3076, 1420),            # 280 MB
    "dx 64, once f32": (F32, [40, 0, 70, 133, 1, 9, 0, 58], 3076, 1420),          # 38 rows a group
    "dx 128, weights once": (F16, [30, 0, 41, 200, 1, 9, 0, 8], 4104, 2056),
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("path", BACKWARD)
def test_backward_tiles(path, wide):
    dtype, m, K, F = BACKWARD[path]
    L = Layer(m, K, F, dtype, bias=False, seed=K)
    h = torch.randn(L.T, 2 * F, generator=torch.Generator().manual_seed(1)).to(dtype)
    dw0 = torch.randn(L.G, 2 * F, K, generator=torch.Generator().manual_seed(2))
    dw = dw0.to(DEV) if wide else L.new(L.G, 2 * F, K).fill_(7.0)
    dh, dx = L.new(L.T, 2 * F), nan_tail(L.T + 1, K, L.T, dtype, DEV)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dw, L.ws, h=h.to(DEV), accumulate=wide)
    check(dh, *grad_limits("silu", to64(h), np.zeros(h.shape), to64(L.da), dtype), "dh")
    x, w, d = to64(L.x), to64(L.w), to64(dh)
    rx, rw, _ = gated.glu_backward(x, w, d, m)
    mx, mw, _ = gated.glu_backward(np.abs(x), np.abs(w), np.abs(d), m)
    check(dx[:L.T], rx, (2 * F + 2) * 2 * V * mx + half_step(dtype, rx), "dx")
    assert torch.isnan(dx[L.T:]).all()
    if wide:
        rw, mw = rw + to64(dw0), mw + np.abs(to64(dw0))
    check(dw, rw, (np.array(m)[:, None, None] + 3) * 2 * V * mw + half_step(F32 if wide else dtype, rw), "dw")


# (type, rows of the groups, K, F): the contraction in two parts of unequal numbers of stages, one part past the end
PARTS = [(BF, [5, 0, 40], 264, 72), (BF, [1], 40, 40), (F16, [9, 2], 136, 264), (F32, [20, 1], 132, 72), (F32, [17], 20, 20)]


@pytest.mark.parametrize("dtype,m,K,F", PARTS, ids=str)
def test_contraction_in_two_parts(dtype, m, K, F):
    for n in (K, K + 32, 5 * K):  # 1 to 42 stages
        L = Layer(m, n, F, dtype, seed=n)
        a, h = nan_tail(L.T + 2, F, L.T, dtype, DEV), L.new(L.T, 2 * F)
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h)
        ref_h, e = L.h()
        check(a[:L.T], *glu_limits("silu", ref_h, e, dtype), "a")
        check(h, ref_h, e + half_step(dtype, ref_h), "h")
        dh, dx, dw = L.new(L.T, 2 * F), nan_tail(L.T + 1, n, L.T, dtype, DEV), L.new(L.G, 2 * F, n)
        gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dw, L.ws, h=h)
        w, d = to64(L.w), to64(dh)
        rx, mx = (gated.glu_backward(to64(L.x), f(w), f(d), m)[0] for f in (np.asarray, np.abs))
        check(dx[:L.T], rx, (2 * F + 2) * 2 * V * mx + half_step(dtype, rx), "dx")
        assert torch.isnan(dx[L.T:]).all() and torch.isnan(a[L.T:]).all()


@pytest.mark.parametrize("K", [16, 128, 144, 272, 1040])
@pytest.mark.parametrize("gate", [None, "silu"])
def test_int8_contraction_in_two_parts(gate, K):
    P = Int8([5, 0, 40], K, 144, F16, seed=K)
    h, e = P.h()
    y = nan_tail(P.T + 2, 72 if gate else 144, P.T, F16, DEV)
    if gate:
        gl.gl_glu_forward_int8(*P.args, y, P.ws, bias=P.bias)
        check(y[:P.T], *glu_limits(gate, h, e, F16), "a")
    else:
        gl.gl_forward_int8(*P.args, y, P.ws, bias=P.bias)
        check(y[:P.T], h, e + half_step(F16, h), "y")
    assert torch.isnan(y[P.T:]).all()


# the largest widths: 2^20 values of a row, or weight rows
@pytest.mark.parametrize("dtype,m", [(BF, [3, 37]), (BF, [300]), (F16, [2]), (F32, [2]), (F32, [3, 270])], ids=str)
@pytest.mark.parametrize("wide", [False, True])
def test_largest_sizes(dtype, m, wide):
    """Outputs and gradients at the first and the last columns."""
    K, F = (16, 1 << 19) if wide else (1 << 20, 8)
    g = torch.Generator(DEV).manual_seed(0)
    T, G = sum(m), len(m)
    x, w, da = (torch.randn(*s, generator=g, device=DEV) for s in ((T, K), (G, 2 * F, K), (T, F)))
    x, w, da = x.to(dtype), (w * K ** -0.5).to(dtype), da.to(dtype)
    ws = gl.new_workspace(G)
    gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), T, ws)
    new = lambda *s: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    a, dh, dx, dw = new(T, F), new(T, 2 * F), new(T, K), new(G, 2 * F, K)
    gl.gl_glu_forward(x, w, a, ws)
    gl.gl_glu_backward(x, w, da, dh, dx, dw, ws)
    for c in (slice(0, 8), slice(F - 8, F)):  # columns of F, with their weight rows
        wc = to64(torch.cat([w[:, :F][:, c], w[:, F:][:, c]], 1))
        x64, dac = to64(x), to64(da[:, c])
        h = gated.product(x64, wc, None, m)
        e = (K + 2) * V * gated.product(np.abs(x64), np.abs(wc), None, m)
        check(a[:, c], *glu_limits("silu", h, e, dtype), "a")
        got = torch.cat([dh[:, :F][:, c], dh[:, F:][:, c]], 1)
        check(got, *grad_limits("silu", h, e, dac, dtype), "dh")
        d = to64(got)
        rw = gated.glu_backward(x64, wc, d, m)[1]
        mw = gated.glu_backward(np.abs(x64), np.abs(wc), np.abs(d), m)[1]
        check(torch.cat([dw[:, :F][:, c], dw[:, F:][:, c]], 1), rw,
              (np.array(m)[:, None, None] + 2) * 2 * V * mw + half_step(dtype, rw), "dw")
    for c in (slice(0, 8), slice(K - 8, K)):
        d, wc = to64(dh), to64(w[:, :, c])
        rx, mx = (gated.glu_backward(to64(x[:, c]), f(wc), f(d), m)[0] for f in (np.asarray, np.abs))
        check(dx[:, c], rx, (2 * F + 2) * 2 * V * mx + half_step(dtype, rx), "dx")
