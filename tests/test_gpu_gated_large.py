"""The gated layer, the quantizer and the 8-bit integer products where element offsets pass 2^32
and where the weights outgrow the last-level cache; and a training step of a gated layer with the layer behind it
(tolerances as in test_gpu_glu.py and test_gpu_int8.py).  Of the large outputs the last rows, or
the last group's matrix, are compared."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import to64
from oracle import gated
from test_gpu_glu import ACTS, TYPES, V, Layer, check, glu_limits, grad_limits, half_step
from test_gpu_int8 import Int8

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
ROWS, WIDE = (1 << 18) + 70, 16400  # a matrix of 2^32 + 21 million elements


def new(*s, dtype=BF):
    return torch.empty(*s, dtype=dtype, device=DEV)


def offsets(m):
    ws = gl.new_workspace(len(m))
    gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), sum(m), ws)
    return ws


@pytest.fixture
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_layer_of_many_rows(memory):
    """h, dh of 2^32 elements and more: forward, both backwards (h kept and not), dx."""
    K, F, last = 8, WIDE // 2, 70
    m = [ROWS - last - 3, 3, last]
    g = torch.Generator(DEV).manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    x, w, b, da, ws = r(ROWS, K), r(3, 2 * F, K), r(3, 2 * F), new(ROWS, F), offsets(m)
    da.zero_()
    da[-last:] = r(last, F)
    a, h = new(ROWS, F), new(ROWS, 2 * F)
    gl.gl_glu_forward(x, w, a, ws, bias=b, h=h)
    x64, w64, b64, m1 = to64(x[-last:]), to64(w[2:]), to64(b[2:]), [last]
    ref_h = gated.product(x64, w64, b64, m1)
    e = (K + 2) * V * gated.product(np.abs(x64), np.abs(w64), np.abs(b64), m1)
    check(h[-last:], ref_h, e + half_step(BF, ref_h), "h")
    check(a[-last:], *glu_limits("silu", ref_h, e, BF), "a")
    dx, a2, dw = new(ROWS, K), new(ROWS, F), new(3, 2 * F, K)
    d64, k64 = to64(da[-last:]), to64(h[-last:])
    for kept in (False, True):
        dh = h if kept else new(ROWS, 2 * F)
        gl.gl_glu_backward(x, w, da, dh, dx, dw, ws, h=h if kept else None, bias=b, a=a2)
        hv, ev = (k64, np.zeros_like(e)) if kept else (ref_h, e)
        check(dh[-last:], *grad_limits("silu", hv, ev, d64, BF), "dh")
        check(a2[-last:], *glu_limits("silu", hv, ev, BF), "a again")
        d = to64(dh[-last:])
        (rx, rw, _), (mx, mw, _) = (gated.glu_backward(f(x64), f(w64), f(d), m1) for f in (np.asarray, np.abs))
        check(dx[-last:], rx, (2 * F + 2) * 2 * V * mx + half_step(BF, rx), "dx")
        check(dw[2:], rw, (last + 2) * 2 * V * mw + half_step(BF, rw), "dw")
        assert not dw[:2].any()  # da is 0 there
        del dh


def test_layer_of_large_weights(memory):
    """Weights and weight gradients of 2^32 elements and more, bf16."""
    G, K, F = 64, 8200, 4104
    m = [2] + [0] * (G - 2) + [9]
    g = torch.Generator(DEV).manual_seed(0)
    x, w, da = (torch.randn(*s, generator=g, device=DEV, dtype=BF) for s in ((11, K), (G, 2 * F, K), (11, F)))
    w *= K ** -0.5
    ws, a, dh, dx = offsets(m), new(11, F), new(11, 2 * F), new(11, K)
    dw = new(G, 2 * F, K).fill_(7.0)
    gl.gl_glu_forward(x, w, a, ws)
    gl.gl_glu_backward(x, w, da, dh, dx, dw, ws)
    x64, w64 = to64(x[2:]), to64(w[-1:])
    h = gated.product(x64, w64, None, [9])
    e = (K + 2) * V * gated.product(np.abs(x64), np.abs(w64), None, [9])
    check(a[2:], *glu_limits("silu", h, e, BF), "a")
    check(dh[2:], *grad_limits("silu", h, e, to64(da[2:]), BF), "dh")
    d = to64(dh[2:])
    rx, rw, _ = gated.glu_backward(x64, w64, d, [9])
    mx, mw, _ = gated.glu_backward(np.abs(x64), np.abs(w64), np.abs(d), [9])
    check(dx[2:], rx, (2 * F + 2) * 2 * V * mx + half_step(BF, rx), "dx")
    check(dw[-1:], rw, (9 + 3) * 2 * V * mw + half_step(BF, rw), "dw")
    assert not dw[1:-1].any()  # groups without rows


def test_int8_of_many_rows(memory):
    """The quantizer's input and codes, the product's rows and outputs, past 2^32 elements."""
    last = 70
    m = [ROWS - last - 3, 3, last]
    x = new(ROWS, WIDE).zero_()
    g = torch.Generator(DEV).manual_seed(0)
    x[-last:] = torch.randn(last, WIDE, generator=g, device=DEV).to(BF)
    q, s = new(ROWS, WIDE, dtype=torch.int8), new(ROWS, dtype=F32)
    gl.gl_quantize_int8(x, q, s)
    rq, rs = gated.quantize_int8(x[-last:].float().cpu().numpy())
    assert np.array_equal(q[-last:].cpu().numpy(), rq) and np.array_equal(s[-last:].cpu().numpy(), rs)
    assert not q[0].any() and s[0] > 0
    del x
    ws = offsets(m)
    for narrow in (True, False):  # long rows and few columns, then the other way round
        K, N = (WIDE, 16) if narrow else (16, WIDE)
        w = torch.randint(-128, 128, (3, N, K), generator=g, device=DEV, dtype=torch.int8)
        wsc = torch.rand(3, N, generator=g, device=DEV)
        xq = q if narrow else q[:, :16].contiguous()
        h = gated.product_int8(*(to64(t) for t in (xq[-last:], s[-last:], w[2:], wsc[2:])), None, [last])
        e = 2.0 ** -21 * np.abs(h)
        y, a = new(ROWS, N), new(ROWS, N // 2)
        gl.gl_forward_int8(xq, s, w, wsc, y, ws)
        check(y[-last:], h, e + half_step(BF, h), "y")
        gl.gl_glu_forward_int8(xq, s, w, wsc, a, ws)
        check(a[-last:], *glu_limits("silu", h, e, BF), "a")


# weights past 256 MB with few rows a group: read once; tiles of 64 and of 128 rows (int8: 256)
@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("dtype", TYPES)
def test_layer_of_weights_past_the_cache(dtype, rows):
    L = Layer([rows, 0, 2 * rows, 1] * 2, 4104, 3528 if dtype != F32 else 1764, dtype, bias=rows == 2)
    a, h = L.new(L.T, L.F), L.new(L.T, 2 * L.F) if rows == 2 else None
    gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h)
    ref_h, e = L.h()
    check(a, *glu_limits("silu", ref_h, e, dtype), "a")
    if h is not None:
        check(h, ref_h, e + half_step(dtype, ref_h), "h")
    dh, dw = L.new(L.T, 2 * L.F), torch.empty_like(L.dw_)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, None, dw, L.ws, bias=L.db_)
    check(dh, *grad_limits("silu", ref_h, e, to64(L.da), dtype), "dh")


@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("name", [None, *ACTS])
def test_int8_weights_past_the_cache(name, rows):
    P = Int8([rows, 0, 2 * rows, 1] * 4, 4112, 4112, BF)
    h, e = P.h()
    y = new(P.T, P.N // 2 if name else P.N)
    if name:
        gl.gl_glu_forward_int8(*P.args, y, P.ws, bias=P.bias, act=ACTS[name])
        check(y, *glu_limits(name, h, e, BF), "a")
    else:
        gl.gl_forward_int8(*P.args, y, P.ws, bias=P.bias)
        check(y, h, e + half_step(BF, h), "y")


# dW on tiles of 64, 128 and 256 rows
@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("m,K,F", [([5, 0, 70], 264, 72), ([700], 1544, 1032), ([3, 0, 129, 66], 2312, 1160)], ids=str)
def test_weight_gradients_added_into_16_bits(m, K, F, dtype):
    """dW + the product, rounded once; a group without rows is left as it was."""
    L = Layer(m, K, F, dtype, bias=False)
    h = torch.randn(L.T, 2 * F, generator=torch.Generator().manual_seed(1)).to(dtype)
    dw0 = torch.randn(L.G, 2 * F, K, generator=torch.Generator().manual_seed(2)).to(dtype)
    dh, dw = L.new(L.T, 2 * F), dw0.to(DEV)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, None, dw, L.ws, h=h.to(DEV), accumulate=True)
    x, w, d = to64(L.x), to64(L.w), to64(dh)
    ref = to64(dw0) + gated.glu_backward(x, w, d, m)[1]
    mag = np.abs(to64(dw0)) + gated.glu_backward(np.abs(x), np.abs(w), np.abs(d), m)[1]
    check(dw, ref, (np.array(m)[:, None, None] + 3) * 2 * V * mag + half_step(dtype, ref), "dw")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [9, 700])
def test_training_step_of_an_expert_layer(T, dtype):
    """y = W2 (silu(W_gate x) * (W_up x)) and its gradients by the calls a training step makes:
    gated forward (h kept or not), second product, its backward, gated backward.  Each call is
    compared with the oracle's step from that call's own inputs."""
    K, F, N = 136, 200, 72
    m = [T - 5, 0, 5]
    for kept in (False, True):
        L = Layer(m, K, F, dtype, bias=True, seed=T)
        g = torch.Generator().manual_seed(1)
        w2, dy = (torch.randn(*s, generator=g).to(dtype) for s in ((3, N, F), (T, N)))
        w2_, dy_ = w2.to(DEV), dy.to(DEV)
        a, h, y = L.new(T, F), L.new(T, 2 * F) if kept else None, L.new(T, N)
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h)
        gl.gl_forward(a, w2_, y, L.ws)
        da, dw2 = L.new(T, F), L.new(3, N, F)
        gl.gl_dgrad(dy_, w2_, da, L.ws)
        gl.gl_wgrad(a, dy_, dw2, L.ws)
        dh, dx, dw, db = L.new(T, 2 * F), L.new(T, K), L.new(3, 2 * F, K), L.new(3, 2 * F)
        gl.gl_glu_backward(L.dx_, L.dw_, da, dh, dx, dw, L.ws, h=h, bias=L.db_, db=db)
        ref_h, e = L.h()
        check(a, *glu_limits("silu", ref_h, e, dtype), "a")
        a64, w64 = to64(a), to64(w2)
        ref_y, mag = gated.product(a64, w64, None, m), gated.product(np.abs(a64), np.abs(w64), None, m)
        check(y, ref_y, (F + 2) * 2 * V * mag + half_step(dtype, ref_y), "y")
        rda, rdw2, _ = gated.glu_backward(a64, w64, to64(dy), m)
        mda, mdw2, _ = gated.glu_backward(np.abs(a64), np.abs(w64), np.abs(to64(dy)), m)
        n = np.array(m)[:, None, None]
        check(da, rda, (N + 2) * 2 * V * mda + half_step(dtype, rda), "da")
        check(dw2, rdw2, (n + 3) * 2 * V * mdw2 + half_step(dtype, rdw2), "dw2")
        if kept:
            ref_h, e = to64(h), np.zeros_like(e)
        check(dh, *grad_limits("silu", ref_h, e, to64(da), dtype), "dh")
        x, w, d = to64(L.x), to64(L.w), to64(dh)
        rx, rw, rb = gated.glu_backward(x, w, d, m)
        mx, mw, mb = gated.glu_backward(np.abs(x), np.abs(w), np.abs(d), m)
        check(dx, rx, (2 * F + 2) * 2 * V * mx + half_step(dtype, rx), "dx")
        check(dw, rw, (n + 3) * 2 * V * mw + half_step(dtype, rw), "dw")
        check(db, rb, (n[..., 0] + 2) * 2 * V * mb + half_step(dtype, rb), "db")
