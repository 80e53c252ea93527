"""Every kernel and tile of the gated layer, of its backward's products and of the 8-bit integer products, at sizes
that take it (test_glu_choice.py, on the CPU, asks the library's rules and holds the labels here to
them), against the float64 oracle (tolerances as in test_gpu_glu.py and test_gpu_int8.py; fp32 sums
as in any order)."""
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
RAGGED = [30, 0, 41, 200, 1, 9, 0, 8]
WIDER = [40, 0, 70, 133, 1, 9, 0, 58]

# kernel: (type, rows of the groups, K, F); a tile as rows by weight rows, "parts": the contraction in two,
# "once": weights past the last-level cache
FORWARD = [
    ("32x32 parts", BF, [5, 0, 40], 264, 72),
    ("32x32 parts", F16, [33, 0, 1, 40], 136, 136),
    ("32x32", BF, [6, 0, 13, 1] * 5, 200, 776),
    ("32x32", F16, [300], 72, 1032),
    ("32x32 once", BF, [5, 0, 17, 1, 0, 3, 8, 6], 2056, 4104),
    ("64x64", BF, [20, 0, 70, 30] * 2, 264, 776),
    ("64x64", F16, [20, 0, 65, 5, 0, 0, 129], 72, 840),
    ("64x64 once", F16, [25, 0, 33, 12, 40, 1, 30, 19], 2072, 4104),
    ("128x128", BF, [30, 20, 0, 200], 136, 3336),
    ("128x128", F16, [30, 20, 0, 200], 200, 3336),
    ("128x128 once", BF, RAGGED, 4104, 2056),
    ("256 ragged", BF, [100, 260, 1], 200, 4104),
    ("256 ragged", F16, [100, 260, 1], 136, 4104),
    ("256 full", BF, [300, 513], 136, 3464),
    ("256 full", F16, [300, 513], 200, 3464),
    ("few", F32, [5, 0, 11], 132, 40),
    ("32x64 parts", F32, [33, 0, 1, 40], 100, 136),
    ("32x64", F32, [33, 0, 1, 40], 100, 2052),
    ("32x64 once", F32, [2, 0, 7, 33, 1, 9, 0, 8], 2052, 2052),
    ("64x64", F32, [300, 2, 513], 132, 1000),
    ("64x64 once", F32, WIDER, 2056, 2052),
    ("256 ragged", F32, [2] * 40, 36, 6660),
    ("256 full", F32, [300, 258], 100, 52432),
]
DX = [
    ("32x64 parts", BF, [33, 0, 1, 70], 264, 72),
    ("32x64 parts", F16, [33, 0, 1, 70], 520, 40),
    ("64x64", BF, [130, 0, 400, 257, 300], 1032, 520),
    ("64x64", F16, [100, 0, 300, 257], 1032, 104),
    ("128x128", BF, [130, 0, 400, 257, 300], 2056, 72),
    ("128x128", F16, [130, 0, 400, 257, 300], 2056, 104),
    ("128x128 once", BF, RAGGED, 4104, 2056),
    ("256 ragged", F16, [3, 0, 20, 1] * 8, 1544, 72),
    ("256 ragged once", F16, [100, 0, 140, 500, 1, 59, 0, 8], 4104, 2056),
    ("256 full", BF, [300, 2, 513], 8200, 40),
    ("32x64 parts", F32, [33, 0, 1, 70], 260, 36),
    ("32x64", F32, [33, 0, 1, 70], 3844, 36),
    ("32x64 once", F32, [2, 0, 7, 33, 1, 9, 0, 8], 4100, 1028),
    ("64x64", F32, [300, 2, 513], 2052, 68),
    ("64x64 once", F32, WIDER, 3204, 1312),
]
DW = [
    ("64x64", BF, [5, 0, 70, 20], 264, 72),
    ("64x64", F16, [5, 0, 70, 20], 264, 72),
    ("128x128", BF, [130, 0, 400, 257, 300], 1032, 520),
    ("128x128", F16, [700], 1544, 1032),
    ("256 full", BF, [3, 0, 129, 0, 66, 1], 2312, 2312),
    ("256 full", F16, [6, 0, 13, 1] * 4, 1032, 520),
    ("256 written once", F16, [20, 0, 33, 1, 0, 3, 8, 6], 4104, 2056),
    ("64x64", F32, [130, 0, 1, 257], 516, 260),
    ("64x64 once", F32, [2, 0, 7, 33, 1, 9, 0, 8], 2052, 2052),
]
# K and the weights' rows N, 2F of the gated product
INT8 = [
    ("32x64 parts", [33, 0, 1, 40], 272, 144),
    ("32x64", [15, 0, 17, 1] * 8, 144, 1056),
    ("32x64 once", [5, 0, 17, 1, 0, 3, 8, 6], 4112, 8208),
    ("128x128", [30, 20, 0, 200], 272, 6672),
    ("128x128 once", [100, 80], 16400, 8208),
    ("256 ragged", [100, 260, 1], 144, 8208),
    ("256 ragged once", RAGGED, 8208, 4112),
    ("256 full", [300, 513], 272, 6928),
]


def some(i, label):
    """Activations: tiles of 256 rows have a kernel for each."""
    names = list(ACTS)
    return names if label.startswith("256") else [names[i % 3]]


@pytest.mark.parametrize("i", range(len(FORWARD)), ids=lambda i: f"{FORWARD[i][0]}-{str(FORWARD[i][1])[6:]}")
def test_forward(i):
    label, dtype, m, K, F = FORWARD[i]
    L = Layer(m, K, F, dtype, seed=i, lists=i % 2 == 1)
    ref_h, e = L.h()
    for name in some(i, label):
        a, h = nan_tail(L.T + 2, F, L.T, dtype, DEV), L.new(L.T, 2 * F)
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h, act=ACTS[name])
        ref, lim = glu_limits(name, ref_h, e, dtype)
        check(a[:L.T], ref, lim, f"a {name}")
        check(h, ref_h, e + half_step(dtype, ref_h), "h")
        assert torch.isnan(a[L.T:]).all()
        dh, a2, dw = L.new(L.T, 2 * F), L.new(L.T, F), L.new(L.G, 2 * F, K)
        gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, None, dw, L.ws, bias=L.db_, a=a2, act=ACTS[name])
        check(a2, ref, lim, f"a again {name}")
        check(dh, *grad_limits(name, ref_h, e, to64(L.da), dtype), f"dh {name}")


def backward(L, i, dx, dw, accumulate):
    """dh from kept values, checked."""
    h = torch.randn(L.T, 2 * L.F, generator=torch.Generator().manual_seed(i)).to(L.dtype)
    dh = L.new(L.T, 2 * L.F)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dw, L.ws, h=h.to(DEV), accumulate=accumulate)
    check(dh, *grad_limits("silu", to64(h), np.zeros(h.shape), to64(L.da), L.dtype), "dh")
    return to64(dh)


@pytest.mark.parametrize("i", range(len(DX)), ids=lambda i: f"{DX[i][0]}-{str(DX[i][1])[6:]}")
def test_dx(i):
    label, dtype, m, K, F = DX[i]
    L = Layer(m, K, F, dtype, bias=False, seed=i, lists=i % 2 == 1)
    dx = nan_tail(L.T + 1, K, L.T, dtype, DEV)
    d = backward(L, i, dx, L.new(L.G, 2 * F, K), False)
    rx, mx = np.zeros((L.T, K)), np.zeros((L.T, K))
    for g, r in gated.groups(m):
        w = to64(L.w[g])
        rx[r], mx[r] = d[r] @ w, np.abs(d[r]) @ np.abs(w)
    check(dx[:L.T], rx, (2 * F + 2) * 2 * V * mx + half_step(dtype, rx), "dx")
    assert torch.isnan(dx[L.T:]).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("i", range(len(DW)), ids=lambda i: f"{DW[i][0]}-{str(DW[i][1])[6:]}")
def test_dw(i, wide):
    label, dtype, m, K, F = DW[i]
    L = Layer(m, K, F, dtype, bias=False, seed=i)
    dw0 = torch.randn(L.G, 2 * F, K, generator=torch.Generator().manual_seed(2)) if wide else None
    dw = dw0.to(DEV) if wide else L.new(L.G, 2 * F, K).fill_(7.0)
    d = backward(L, i, None, [v for v in dw] if i % 2 else dw, wide)
    x = to64(L.x)
    for g, r in gated.groups(m):
        ref, mag = d[r].T @ x[r], np.abs(d[r]).T @ np.abs(x[r])
        if wide:
            old = to64(dw0[g])
            ref, mag = ref + old, mag + np.abs(old)
        check(dw[g], ref, (m[g] + 3) * 2 * V * mag + half_step(F32 if wide else dtype, ref), f"dw {g}")


@pytest.mark.parametrize("i", range(len(INT8)), ids=lambda i: INT8[i][0])
def test_int8(i):
    label, m, K, N = INT8[i]
    P = Int8(m, K, N, F32, seed=i, bias=False, lists=i % 2 == 1)
    h, e = P.h()
    for out in (BF, F16, F32):
        y = nan_tail(P.T + 2, N, P.T, out, DEV)
        gl.gl_forward_int8(*P.args, y, P.ws)
        check(y[:P.T], h, e + half_step(out, h), f"y {out}")
        assert torch.isnan(y[P.T:]).all()
        for name in some(i, label):
            a = nan_tail(P.T + 2, N // 2, P.T, out, DEV)
            gl.gl_glu_forward_int8(*P.args, a, P.ws, act=ACTS[name])
            check(a[:P.T], *glu_limits(name, h, e, out), f"a {out} {name}")
            assert torch.isnan(a[P.T:]).all()
