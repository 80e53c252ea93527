"""Refusals of the gated layer's and the 8-bit integer product's entry points: each call fails
its checks on the host before anything is enqueued (no pointer is dereferenced)."""
import os

import pytest
import torch

import grouped_gemm_gl_amd as gl

pytestmark = pytest.mark.skipif(not os.path.exists(gl.library_path), reason="library not built")

A, B, C_, D, E_, F_ = (0x100000 * i for i in range(1, 7))  # aligned, never dereferenced
F32, BF16, F16, MX = gl.GL_F32, gl.GL_BF16, gl.GL_F16, gl.GL_E4M3

GLU = dict(G=4, K=64, F=32, T=3, dt=BF16, act=0, x=A, w=B, wp=None, b=None, bp=None, h=None, a=C_, rows=3, ws=D)
SIZES = [(dict(G=0), -1), (dict(K=0), -1), (dict(F=0), -1), (dict(F=-8), -1), (dict(T=-1), -1), (dict(dt=MX), -2),
         (dict(dt=7), -2), (dict(act=3), -1), (dict(act=-1), -1), (dict(K=60), -3), (dict(F=36), -3),
         (dict(dt=F32, K=62), -3), (dict(dt=F32, F=30), -3), (dict(K=(1 << 20) + 8), -3), (dict(F=(1 << 19) + 8), -3),
         (dict(T=1 << 31, rows=1 << 31), -3), (dict(ws=None), -1), (dict(ws=D + 8), -1), (dict(w=None), -1),
         (dict(wp=B), -1), (dict(w=B + 8), -1), (dict(w=None, wp=B + 4), -1), (dict(b=E_, bp=E_), -1),
         (dict(b=E_ + 2), -1), (dict(x=None), -1), (dict(x=A + 2), -1)]


@pytest.mark.parametrize("kw,code", SIZES + [(dict(rows=2), -3), (dict(a=None), -1), (dict(a=C_ + 8), -1),
                                             (dict(h=E_ + 4), -1), (dict(h=C_), -1)])
def test_glu_forward_refuses(kw, code):
    assert gl.load().gl_glu_forward(*{**GLU, **kw}.values(), None) == code and gl.load().gl_last_error()


GLU_B = dict(G=4, K=64, F=32, T=3, dt=BF16, wdt=BF16, act=0, x=A, w=B, wp=None, b=None, bp=None, h=None, da=C_, dh=E_,
             a=None, dx=F_, rows=3, dw=A, dwp=None, db=None, dbp=None, acc=0, ws=D)


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in SIZES if "dt" not in k or k["dt"] != F32] + [
    (dict(dt=F32, wdt=F32, K=62), -3), (dict(dt=F32, wdt=F32, F=30), -3), (dict(wdt=F16), -2), (dict(wdt=MX), -2),
    (dict(da=None), -1), (dict(da=C_ + 8), -1), (dict(dh=None), -1), (dict(dh=E_ + 4), -1), (dict(dh=C_), -1),
    (dict(h=B + 8), -1), (dict(a=B + 8), -1), (dict(a=E_), -1), (dict(a=C_), -1), (dict(dx=F_ + 8), -1),
    (dict(rows=2), -3), (dict(dw=None), -1), (dict(dwp=A), -1), (dict(dw=A + 8), -1), (dict(db=A, dbp=A), -1),
    (dict(db=A + 2), -1), (dict(acc=2), -1),
])
def test_glu_backward_refuses(kw, code):
    assert gl.load().gl_glu_backward(*{**GLU_B, **kw}.values(), None) == code and gl.load().gl_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(cols=0), -1), (dict(cols=-16), -1), (dict(dt=MX), -2), (dict(cols=24), -3),
    (dict(cols=(1 << 22) + 16), -3), (dict(rows=1 << 31), -3), (dict(src=None), -1), (dict(src=A + 2), -1),
    (dict(data=None), -1), (dict(data=B + 8), -1), (dict(scale=None), -1), (dict(scale=C_ + 2), -1), (dict(data=A), -1),
])
def test_quantize_int8_refuses(kw, code):
    args = {**dict(rows=3, cols=64, dt=BF16, src=A, data=B, scale=C_), **kw}
    assert gl.load().gl_quantize_int8(*args.values(), None) == code and gl.load().gl_last_error()


INT8 = dict(G=4, K=64, F=32, T=3, dt=BF16, x=A, xs=B, w=C_, wp=None, s=D, sp=None, b=None, bp=None, y=E_, rows=3, ws=F_)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(G=0), -1), (dict(K=0), -1), (dict(F=0), -1), (dict(T=-1), -1), (dict(dt=MX), -2), (dict(K=72), -3),
    (dict(F=28), -3), (dict(K=1 << 17), -3), (dict(F=(1 << 20) + 8), -3), (dict(rows=2), -3), (dict(ws=None), -1),
    (dict(ws=F_ + 4), -1), (dict(w=None, s=None), -1), (dict(wp=C_), -1), (dict(w=C_ + 8), -1), (dict(s=None), -1),
    (dict(s=None, sp=D), -1), (dict(s=D + 2), -1), (dict(w=None, wp=C_, s=None, sp=D + 4), -1), (dict(b=A, bp=A), -1),
    (dict(b=A + 8), -1), (dict(x=None), -1), (dict(x=A + 4), -1), (dict(xs=None), -1), (dict(xs=B + 1), -1),
    (dict(y=None), -1), (dict(y=E_ + 4), -1), (dict(T=1 << 31, rows=1 << 31), -3),
])
def test_int8_products_refuse(gated, kw, code):
    v = list({**INT8, **kw}.values())
    if gated:
        rc = gl.load().gl_glu_forward_int8(*v[:5], 0, *v[5:], None)
    else:
        rc = gl.load().gl_forward_int8(*v, None)
    assert rc == code and gl.load().gl_last_error()


def test_gated_int8_refuses_an_unknown_activation():
    v = list(INT8.values())
    assert gl.load().gl_glu_forward_int8(*v[:5], 5, *v[5:], None) == -1


def test_no_rows_is_no_error():
    ok = lambda d, **kw: {**d, **kw}.values()  # noqa: E731
    lib = gl.load()
    assert lib.gl_glu_forward(*ok(GLU, T=0, rows=0, x=None, a=None), None) == 0
    assert lib.gl_forward_int8(*ok(INT8, T=0, rows=0, x=None, xs=None, y=None), None) == 0
    assert lib.gl_quantize_int8(0, 64, BF16, None, None, None, None) == 0


def test_binding_refuses_before_the_library():
    """Shapes, types and devices that do not agree (CPU tensors: nothing runs)."""
    bf, ws = torch.bfloat16, torch.empty(16, dtype=torch.uint8)
    x, w, a = torch.empty(3, 64, dtype=bf), torch.empty(2, 32, 64, dtype=bf), torch.empty(3, 16, dtype=bf)
    q = lambda t: torch.empty(t.shape, dtype=torch.int8)  # noqa: E731
    xs, wsc = torch.empty(3), torch.empty(2, 32)
    bad = [
        lambda: gl.gl_glu_forward(x, w, a, ws),  # not on the GPU
        lambda: gl.gl_glu_forward(x[:, :56], w, a, ws),
        lambda: gl.gl_glu_forward(x, w[:, :31], a, ws),
        lambda: gl.gl_glu_forward(x, w.half(), a, ws),
        lambda: gl.gl_glu_forward(x, w, a.float(), ws),
        lambda: gl.gl_glu_forward(x, w, torch.empty(3, 32, dtype=bf), ws),
        lambda: gl.gl_glu_forward(x, [w[0], w[1, :30]], a, ws),
        lambda: gl.gl_glu_forward(x, w, a, ws, bias=torch.empty(2, 16, dtype=bf)),
        lambda: gl.gl_glu_forward(x, w, a, ws, h=torch.empty(3, 16, dtype=bf)),
        lambda: gl.gl_glu_backward(x, w, a, torch.empty(3, 16, dtype=bf), None, w, ws),
        lambda: gl.gl_glu_backward(x, w, a, torch.empty(3, 32, dtype=bf), x[:, :8], w, ws),
        lambda: gl.gl_glu_backward(x, w, a, torch.empty(3, 32, dtype=bf), None, w[:1], ws),
        lambda: gl.gl_quantize_int8(x, q(x)[:2], xs),
        lambda: gl.gl_quantize_int8(x, torch.empty(3, 64, dtype=torch.uint8), xs),
        lambda: gl.gl_quantize_int8(x, q(x), xs[:2]),
        lambda: gl.gl_forward_int8(q(x), xs[:2], q(w), wsc, torch.empty(3, 32), ws),
        lambda: gl.gl_forward_int8(q(x), xs, q(w), wsc, torch.empty(3, 16), ws),
        lambda: gl.gl_forward_int8(q(x), xs, q(w), [wsc[0], wsc[1]], torch.empty(3, 32), ws),
        lambda: gl.gl_forward_int8(x, xs, w, wsc, torch.empty(3, 32), ws),
        lambda: gl.gl_glu_forward_int8(q(x), xs, q(w), wsc[:, :16], torch.empty(3, 16), ws),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
