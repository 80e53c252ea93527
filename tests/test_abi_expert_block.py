"""Refusals of the norm, routing and few-token entry points: each call fails its checks
on the host before anything is enqueued (no pointer is dereferenced)."""
import os

import pytest
import torch

import grouped_gemm_gl_amd as gl

pytestmark = pytest.mark.skipif(not os.path.exists(gl.library_path), reason="library not built")

A, B, C_, D, E_ = (0x100000 * i for i in range(1, 6))  # aligned, never dereferenced
F32, BF16, F16, MX = gl.GL_F32, gl.GL_BF16, gl.GL_F16, gl.GL_E4M3


def norm(T=4, C=64, dt=BF16, gdt=BF16, x=A, r=None, g=B, eps=1e-6, h=None, y=C_, data=None, scale=None):
    return gl.load().gl_rmsnorm_forward(T, C, dt, gdt, x, r, g, eps, h, y, data, scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(C=0), -1), (dict(dt=MX, gdt=MX), -2), (dict(dt=9, gdt=9), -2), (dict(gdt=F16), -2),
    (dict(dt=F32, gdt=BF16), -2), (dict(C=60), -3), (dict(dt=F32, gdt=F32, C=62), -3), (dict(C=(1 << 22) + 8), -3),
    (dict(T=1 << 31), -3), (dict(g=None), -1), (dict(g=B + 4), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(x=None), -1), (dict(x=A + 2), -1),
    (dict(r=A + 8), -1), (dict(h=A + 8), -1), (dict(y=A + 8), -1), (dict(y=None), -1), (dict(data=D), -1),
    (dict(scale=D), -1), (dict(C=72, data=D, scale=E_), -3), (dict(data=D + 8, scale=E_), -1),
])
def test_rmsnorm_forward_refuses(kw, code):
    assert norm(**kw) == code and gl.load().gl_last_error()


def norm_b(T=4, C=64, dt=BF16, gdt=BF16, dy=A, dh=None, h=B, g=C_, eps=1e-6, dx=D, ddt=F32, dg=E_, acc=0, ws=A):
    return gl.load().gl_rmsnorm_backward(T, C, dt, gdt, dy, dh, h, g, eps, dx, ddt, dg, acc, ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(C=60), -3), (dict(gdt=F16), -2), (dict(ddt=F16), -2), (dict(ddt=MX), -2),
    (dict(acc=2), -1), (dict(ws=None), -1), (dict(ws=A + 8), -1), (dict(dg=E_ + 4), -1), (dict(dy=None), -1),
    (dict(h=None), -1), (dict(dx=None), -1), (dict(dx=D + 8), -1), (dict(dh=A + 8), -1), (dict(eps=-0.5), -1),
])
def test_rmsnorm_backward_refuses(kw, code):
    assert norm_b(**kw) == code and gl.load().gl_last_error()


def route(T=4, E=8, k=2, dt=F32, score=0, renorm=1, l=A, ids=B, w=C_, m=None, ri=None, si=None, ws=None):
    return gl.load().gl_route_forward(T, E, k, dt, score, renorm, l, ids, w, m, ri, si, ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(k=0), -1), (dict(k=9), -3), (dict(E=1025), -3), (dict(E=64, k=33), -3),
    (dict(T=1 << 31), -3), (dict(dt=MX), -2), (dict(score=2), -1), (dict(renorm=2), -1), (dict(l=None), -1),
    (dict(ids=None), -1), (dict(w=C_ + 4), -1), (dict(m=D), -1), (dict(ri=D), -1),
    (dict(m=D, ri=D, si=E_), -1), (dict(m=D + 4, ri=D, si=E_, ws=A), -1), (dict(m=D, ri=D, si=E_, ws=A + 8), -1),
    (dict(m=D, ri=D + 4, si=E_, ws=A), -1),
])
def test_route_forward_refuses(kw, code):
    assert route(**kw) == code and gl.load().gl_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(k=9), -3), (dict(score=-1), -1), (dict(dlogits=None), -1), (dict(dw=B + 4), -1),
    (dict(dt=MX), -2),
])
def test_route_backward_refuses(kw, code):
    a = dict(T=4, E=8, k=2, dt=F32, score=0, renorm=1, l=A, ids=B, dw=C_, dlogits=D)
    a.update(kw)
    assert gl.load().gl_route_backward(*a.values(), None) == code and gl.load().gl_last_error()


MOE = dict(E=4, K=64, F=32, N=64, T=3, k=2, dt=BF16, wdt=BF16, x=A, ids=B, w=C_, w1=A, w1p=None, s1=None, s1p=None,
           b1=None, b1p=None, w2=B, w2p=None, s2=None, s2p=None, b2=None, b2p=None, res=None, y=D, rows=3, ws=E_)


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), -1), (dict(K=0), -1), (dict(F=0), -1), (dict(N=-8), -1), (dict(T=-1), -1), (dict(k=0), -1),
    (dict(T=65, rows=65), -3), (dict(k=33), -3), (dict(dt=MX, wdt=MX), -2), (dict(wdt=F16), -2),
    (dict(dt=F16, wdt=MX, s1=A, s2=A), -2), (dict(K=60), -3), (dict(F=36), -3), (dict(N=36), -3),
    (dict(wdt=MX, s1=A, s2=A, K=80), -3), (dict(wdt=MX, s1=A, s2=A, F=40), -3), (dict(K=(1 << 22) + 8), -3),
    (dict(T=64, rows=64, k=32, F=1 << 18), -3), (dict(rows=2), -3), (dict(w1=None), -1), (dict(w1p=A), -1),
    (dict(w2=None), -1), (dict(w2=B + 8), -1), (dict(b1=A, b1p=A), -1), (dict(b2=A + 2), -1), (dict(s1=A), -1),
    (dict(wdt=MX), -1), (dict(wdt=MX, s1=A), -1), (dict(wdt=MX, s1=A + 2, s2=A), -1), (dict(wdt=MX, s1p=A, s2=A), -1),
    (dict(x=None), -1), (dict(y=None), -1), (dict(ws=None), -1), (dict(ws=E_ + 8), -1), (dict(res=A + 8), -1),
    (dict(ids=None), -1), (dict(w=C_ + 2), -1), (dict(w1=None, w1p=A + 4), -1),
])
def test_moe_few_tokens_refuses(kw, code):
    a = dict(MOE)
    a.update(kw)
    assert gl.load().gl_moe_few_tokens(*a.values(), None) == code and gl.load().gl_last_error()


def test_nothing_to_do_and_workspace_sizes():
    assert norm(T=0, x=None) == 0 and norm_b(T=0, dg=None, dy=None, h=None, dx=None, ws=None) == 0
    assert route(T=0, l=None, ids=None, w=None) == 0
    a = dict(MOE, T=0, x=None, ids=None, w=None, y=None, rows=0, ws=None)
    assert gl.load().gl_moe_few_tokens(*a.values(), None) == 0
    assert gl.gl_rmsnorm_workspace_size(-1, 8) == 0 and gl.gl_rmsnorm_workspace_size(4, 0) == 0
    assert gl.gl_route_workspace_size(-1, 8) == 0 and gl.gl_moe_few_tokens_workspace_size(4, 0, 8, 8) == 0
    for T in (0, 1, 63, 64, 65, 100000):
        assert gl.gl_rmsnorm_workspace_size(T, 4096) >= 16 and gl.gl_route_workspace_size(T, 256) >= 16
        assert gl.gl_rmsnorm_workspace_size(T, 4096) % 16 == 0 and gl.gl_route_workspace_size(T, 256) % 16 == 0
    assert gl.gl_moe_few_tokens_workspace_size(5, 2, 8, 128) >= 5 * 2 * 128 * 4


def test_binding_refuses_on_the_host():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)  # noqa: E731
    x, g = z(3, 64), z(64)
    with pytest.raises(ValueError, match="on the GPU"):
        gl.gl_rmsnorm_forward(x, g, 1e-6, y=z(3, 64))
    for bad in (dict(y=z(3, 32)), dict(y=z(3, 64, d=torch.float32)), dict(data=z(3, 64), scale=z(3, 2)),
                dict(data=z(3, 64, d=torch.uint8), scale=z(3, 3, d=torch.uint8)), dict(residual=z(2, 64), y=z(3, 64))):
        with pytest.raises(ValueError):
            gl.gl_rmsnorm_forward(x, g, 1e-6, **bad)
    with pytest.raises(ValueError):
        gl.gl_rmsnorm_forward(x, z(32), 1e-6, y=z(3, 64))
    with pytest.raises(ValueError, match="workspace"):
        gl.gl_rmsnorm_backward(x, x, g, 1e-6, z(3, 64), dgamma=z(64))
    l, ids, w = z(3, 8, d=torch.float32), z(3, 2, d=torch.int32), z(3, 2, d=torch.float32)
    with pytest.raises(ValueError):
        gl.gl_route_forward(l, ids.long(), w)
    with pytest.raises(ValueError):
        gl.gl_route_forward(l, ids, w, m_splits=z(8, d=torch.int64))
    with pytest.raises(ValueError):
        gl.gl_route_backward(l, ids, w, z(3, 9, d=torch.float32))
    w1, w2, y = z(4, 64, 64), z(4, 64, 32), z(3, 64)
    ws = z(1 << 16, d=torch.uint8)
    with pytest.raises(ValueError, match="on the GPU"):
        gl.gl_moe_few_tokens(x, ids, w, w1, w2, y, ws)
    for bad in (dict(w2=z(4, 64, 48)), dict(w2=z(3, 64, 32)), dict(w2=z(4, 64, 32, d=torch.float16)),
                dict(y=z(3, 72)), dict(workspace=z(64, d=torch.uint8)), dict(ids=ids.long()),
                dict(w1=[w1[0]] * 3, w2=list(w2))):
        a = dict(x=x, ids=ids, weights=w, w1=w1, w2=w2, y=y, workspace=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            gl.gl_moe_few_tokens(**a)
    with pytest.raises(ValueError):
        gl.gl_moe_few_tokens(x, ids, w, w1, w2, y, ws, b1=z(4, 63))


def test_rmsnorm_forward_refuses_one_buffer_for_h_and_y():
    assert norm(h=C_, y=C_) == -1 and "same buffer" in gl.load().gl_last_error().decode()
    assert norm(T=0, x=None, h=C_, y=C_) == 0  # no rows: nothing to write
