"""The gated layer and the 8-bit integer products at sizes that take each of their kernels (split
contraction for few rows and columns, tiles of 64, 128 and 256 rows, the latter with and without
skipped row blocks, several and more than 64 tiles a workgroup), with row lengths that end
inside a stage and stage counts odd and even, against the float64 oracle (tolerances as in
test_gpu_glu.py and test_gpu_int8.py)."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import nan_tail, to64
from oracle import gated
from test_gpu_glu import ACTS, Layer, check, glu_limits, grad_limits, half_step
from test_gpu_int8 import Int8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# kernel: (rows of the groups, F) of the 16-bit layers and K
SHAPES = {
    "few": ([5, 0, 11], 40, (72, 200, 1032)),
    "rows64": ([5, 0, 70, 20], 136, (72, 200, 264)),
    "rows128": ([30, 20, 0, 200], 3336, (40, 136, 200)),
    "rows256_skip": ([100, 260, 1], 4104, (40, 136, 200)),
    "rows256": ([300, 513], 3464, (40, 136, 200)),
}


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("path", SHAPES)
def test_layer_16(path, dtype, name):
    m, F, Ks = SHAPES[path]
    for i, K in enumerate(Ks):
        L = Layer(m, K, F, dtype, bias=i != 1, seed=i)
        a, h = nan_tail(L.T + 2, F, L.T, dtype, DEV), L.new(L.T, 2 * F) if i else None
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h, act=ACTS[name])
        ref_h, e = L.h()
        check(a[:L.T], *glu_limits(name, ref_h, e, dtype), f"a {K}")
        assert torch.isnan(a[L.T:]).all()
        if h is not None:
            check(h, ref_h, e + half_step(dtype, ref_h), f"h {K}")
        dh, a2, dw = L.new(L.T, 2 * F), L.new(L.T, F) if i else None, L.new(L.G, 2 * F, K)
        gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, None, dw, L.ws, bias=L.db_, a=a2, act=ACTS[name])
        check(dh, *grad_limits(name, ref_h, e, to64(L.da), dtype), f"dh {K}")
        if a2 is not None:
            check(a2, *glu_limits(name, ref_h, e, dtype), f"a again {K}")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m,F,K", [([5, 0, 11], 40, 132), ([5, 0, 70, 20], 136, 100), ([2] * 40, 6660, 36),
                                   ([1, 3, 0, 300] * 10, 6660, 68), ([1] * 200, 11524, 8)], ids=str)
def test_layer_f32(m, F, K, name):
    """The last two: tiles of 256 rows, about 8 and 71 of them a workgroup."""
    L = Layer(m, K, F, F32, seed=K)
    a, h = nan_tail(L.T + 2, F, L.T, F32, DEV), L.new(L.T, 2 * F)
    gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h, act=ACTS[name])
    ref_h, e = L.h()
    check(a[:L.T], *glu_limits(name, ref_h, e, F32), "a")
    check(h, ref_h, e + half_step(F32, ref_h), "h")
    assert torch.isnan(a[L.T:]).all()
    if L.T > 1000:
        return
    dh, dw, a2 = L.new(L.T, 2 * F), L.new(L.G, 2 * F, K), L.new(L.T, F)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, None, dw, L.ws, bias=L.db_, a=a2, act=ACTS[name])
    check(dh, *grad_limits(name, ref_h, e, to64(L.da), F32), "dh")
    check(a2, *glu_limits(name, ref_h, e, F32), "a again")


@pytest.mark.parametrize("out", [BF, F16, F32])
@pytest.mark.parametrize("gate", [None, *ACTS])
@pytest.mark.parametrize("path", SHAPES)
def test_int8(path, gate, out):
    m, F, Ks = SHAPES[path]
    for i, K in enumerate(Ks):
        K = (2 * K + 15) // 16 * 16  # the same stages; 80 and 272 end inside one
        N = 2 * F
        P = Int8(m, K, N, out, seed=i, bias=i != 1)
        y = nan_tail(P.T + 2, F if gate else N, P.T, out, DEV)
        h, e = P.h()
        if gate:
            gl.gl_glu_forward_int8(*P.args, y, P.ws, bias=P.bias, act=ACTS[gate])
            check(y[:P.T], *glu_limits(gate, h, e, out), f"a {K}")
        else:
            gl.gl_forward_int8(*P.args, y, P.ws, bias=P.bias)
            check(y[:P.T], h, e + half_step(out, h), f"y {K}")
        assert torch.isnan(y[P.T:]).all()


def test_rows_past_the_group_and_columns_past_the_matrix_read_nothing():
    """NaN in the neighbouring groups' rows and weights, at tiles that end inside: none arrives."""
    m, F, K = [100, 260, 1], 4104, 136
    L = Layer(m, K, F, BF, bias=False)
    want = L.new(L.T, F)
    gl.gl_glu_forward(L.dx_, L.dw_, want, L.ws)
    x, w = L.dx_.clone(), L.dw_.clone()
    x[:100], x[360:], w[0], w[2] = [float("nan")] * 4
    got = L.new(L.T, F)
    gl.gl_glu_forward(x, w, got, L.ws)
    assert torch.equal(got[100:360], want[100:360]) and torch.isnan(got[:100]).all() and torch.isnan(got[360:]).all()


def test_every_split_of_the_rows_gives_the_same_rows():
    """A row's output depends on its own group alone, whatever kernel and tile it meets."""
    K, F = 136, 4104
    L = Layer([361], K, F, BF, bias=False)
    ref_h, e = L.h()
    for m in ([361], [0, 361], [1, 360], [120, 120, 121], [40] * 9 + [1]):
        ws = gl.new_workspace(len(m))
        gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), 361, ws)
        a = L.new(361, F)
        gl.gl_glu_forward(L.dx_, [L.dw_[0]] * len(m), a, ws)
        check(a, *glu_limits("silu", ref_h, e, BF), str(m))


# products of the backward: (rows of the groups, K, F) by the tiles that dx and dW take
BACK = {
    "64": ([5, 0, 70, 20], 264, 72),
    "128": ([130, 0, 400, 257, 300], 1032, 520),        # dx by 128 (144 tiles of 256 rows); dW by 256
    "dw128": ([700], 1544, 1032),                      # dW by 128 (63 tiles of 256)
    "dw256": ([3, 0, 129, 0, 66, 1], 2312, 2312),      # dW over 1000 tiles of 256
    "dx256": ([300, 2, 513], 8200, 40),                # dx 231 tiles of 256, whole
    "dx256_skip": ([3, 0, 20, 1] * 8, 1544, 72),       # and of few rows
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("path", BACK)
def test_backward_products(path, dtype, wide):
    m, K, F = BACK[path]
    L = Layer(m, K, F, dtype, bias=False, seed=K)
    h = torch.randn(L.T, 2 * F, generator=torch.Generator().manual_seed(1)).to(dtype)
    dw0 = torch.randn(L.G, 2 * F, K, generator=torch.Generator().manual_seed(2))
    dw = dw0.to(DEV) if wide else L.new(L.G, 2 * F, K)
    dh, dx, db = L.new(L.T, 2 * F), nan_tail(L.T + 1, K, L.T, dtype, DEV), L.new(L.G, 2 * F)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, [v for v in dw] if wide else dw, L.ws, h=h.to(DEV), db=db,
                       accumulate=wide)
    check(dh, *grad_limits("silu", to64(h), np.zeros(h.shape), to64(L.da), dtype), "dh")
    x, w, d = to64(L.x), to64(L.w), to64(dh)
    rx, rw, rb = gated.glu_backward(x, w, d, m)
    mx, mw, mb = gated.glu_backward(np.abs(x), np.abs(w), np.abs(d), m)
    n = np.array(m)[:, None, None]
    v = 2.0 ** -23
    check(dx[:L.T], rx, (2 * F + 2) * v * mx + half_step(dtype, rx), "dx")
    assert torch.isnan(dx[L.T:]).all()
    if wide:
        rw, mw = rw + to64(dw0), mw + np.abs(to64(dw0))
    check(dw, rw, (n + 3) * v * mw + half_step(F32 if wide else dtype, rw), "dw")
    check(db, rb, (n[..., 0] + 2) * v * mb + half_step(dtype, rb), "db")


def test_backward_products_f32():
    m, K, F = [130, 0, 1, 257], 516, 260
    L = Layer(m, K, F, F32, bias=False, seed=3)
    h = torch.randn(L.T, 2 * F, generator=torch.Generator().manual_seed(1))
    dw, dh, dx = L.new(L.G, 2 * F, K), L.new(L.T, 2 * F), L.new(L.T, K)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dw, L.ws, h=h.to(DEV))
    x, w, d = to64(L.x), to64(L.w), to64(dh)
    rx, rw, _ = gated.glu_backward(x, w, d, m)
    mx, mw, _ = gated.glu_backward(np.abs(x), np.abs(w), np.abs(d), m)
    v = 2.0 ** -24
    check(dx, rx, (2 * F + 2) * v * mx + half_step(F32, rx), "dx")
    check(dw, rw, (np.array(m)[:, None, None] + 2) * v * mw + half_step(F32, rw), "dw")


def test_backward_keeps_nan_in_its_group():
    """Rows and weights of other groups that are NaN reach neither product of a group."""
    m, K, F = [30, 41, 9], 264, 72
    L = Layer(m, K, F, BF, bias=False)
    h = torch.randn(L.T, 2 * F, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    outs = []
    for bad in (False, True):
        x, w, da = L.dx_.clone(), L.dw_.clone(), L.dda.clone()
        if bad:
            x[:30], x[71:], w[0], w[2], da[:30], da[71:] = [float("nan")] * 6
        dh, dx, dw = L.new(L.T, 2 * F), L.new(L.T, K), L.new(3, 2 * F, K)
        gl.gl_glu_backward(x, w, da, dh, dx, dw, L.ws, h=h)
        outs.append((dx, dw))
    assert torch.equal(outs[0][0][30:71], outs[1][0][30:71]) and torch.equal(outs[0][1][1], outs[1][1][1])
    assert torch.isnan(outs[1][0][:30]).all() and torch.isnan(outs[1][1][0]).all()
