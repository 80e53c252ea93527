"""The gated grouped layer (gl_glu_forward, gl_glu_backward) against the float64 oracle.

Tolerances, element by element, with u = finfo.eps / 2 of the type (a rounding is off by at most
that, relative to the value) and v = 2^-24, fp32's:
  h    a sum of K products in fp32, in any order: E_h = (K + 2) v (sum |x w| + |b|)
  a    act' is at most 1.13, so a is off by 1.13 E_g |u| + |act(g)| E_u + E_g E_u, plus the
       activation's own arithmetic, 2^-20 (|act(g)| + 1) |u|, plus u |a| for the rounding
  dh   likewise from h exact (kept) or off by E_h (computed again; act'' is at most 1.13, |act'| too)
  dx, dw, db   the products of dh as it was rounded: the oracle's dh's error through |w|, |x|,
       plus the sum's own error over n terms, (n + 2) 2 v sum |..| (the bias gradient's pairwise
       adds may be off by a whole step), plus u |value|
Values that a 16-bit type holds as subnormals are off by up to half of its smallest step.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import assert_bits_equal, nan_tail, to64
from oracle import gated

pytestmark = pytest.mark.gpu
DEV, V = "cuda", 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
ACTS = {"silu": gl.GL_GLU_SILU, "gelu": gl.GL_GLU_GELU, "gelu_tanh": gl.GL_GLU_GELU_TANH}


def half_step(t, ref):
    f = torch.finfo(t)
    return f.eps / 2 * np.abs(ref) + f.smallest_normal * f.eps / 2


def check(got, ref, lim, what):
    g = to64(got)
    assert g.shape == ref.shape, what
    bad = ~(np.abs(g - ref) <= lim)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) / np.maximum(lim, 1e-300), 0)), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; at {i}: got {g[i]!r}, ref {ref[i]!r}, "
                             f"allowed {lim[i]!r}")


class Layer:
    def __init__(self, m, K, F, dtype, bias=True, seed=0, lists=False, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        G, T = len(m), int(sum(m))
        self.m, self.G, self.T, self.K, self.F, self.dtype = m, G, T, K, F, dtype
        self.x, self.w = (scale * r(T, K)).to(dtype), (r(G, 2 * F, K) * K ** -0.5).to(dtype)
        self.b = (0.5 * r(G, 2 * F)).to(dtype) if bias else None
        self.da = r(T, F).to(dtype)
        self.ws = gl.new_workspace(G)
        gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), T, self.ws)
        dev = (lambda t: None if t is None else [v.to(DEV) for v in t]) if lists else (lambda t: None if t is None else t.to(DEV))
        self.dw_, self.db_ = dev(self.w), dev(self.b)
        self.dx_, self.dda = self.x.to(DEV), self.da.to(DEV)

    def new(self, *s, dtype=None):
        return torch.empty(*s, dtype=dtype or self.dtype, device=DEV)

    def h(self):
        """(h, E_h) in float64."""
        x, w, b = (None if t is None else to64(t) for t in (self.x, self.w, self.b))
        h = gated.product(x, w, b, self.m)
        mag = gated.product(np.abs(x), np.abs(w), None if b is None else np.abs(b), self.m)
        return h, (self.K + 2) * V * mag


def glu_limits(name, h, e, dtype):
    F = h.shape[1] // 2
    g, u, eg, eu = h[:, :F], h[:, F:], e[:, :F], e[:, F:]
    ref = gated.glu(name, h)
    act = np.abs(gated.act(name, g))
    own = 2.0 ** -20 * (act + 1) * np.abs(u)
    return ref, 1.13 * eg * np.abs(u) + (act + own) * eu + eg * eu + own + half_step(dtype, ref)


def grad_limits(name, h, e, da, dtype):
    F = h.shape[1] // 2
    g, u, eg, eu = h[:, :F], h[:, F:], e[:, :F], e[:, F:]
    ref = gated.glu_grad(name, h, da)
    d, s, act = np.abs(da), np.abs(gated.slope(name, g)), np.abs(gated.act(name, g))
    own = 2.0 ** -20
    lim = np.concatenate([d * (np.abs(u) * (1.13 * eg + own * (s + 1)) + (s + own) * eu + 1.13 * eg * eu),
                          d * (1.13 * eg + own * (act + 1))], 1)
    return ref, lim + half_step(dtype, ref)


SPLITS = [[1], [0, 3, 0], [16, 17, 1], [64, 0, 65, 5], [130, 257, 0, 40], [300]]
SIZES = {torch.bfloat16: [(8, 8), (40, 24), (128, 120), (200, 136), (328, 264)],
         torch.float16: [(16, 16), (72, 88), (264, 200)],
         torch.float32: [(4, 4), (36, 20), (100, 132), (160, 260)]}


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", SPLITS, ids=str)
def test_forward(m, dtype, name):
    for i, (K, F) in enumerate(SIZES[dtype]):
        L = Layer(m, K, F, dtype, bias=i % 2 == 0, seed=i, lists=i % 3 == 1)
        a = nan_tail(L.T + 3, F, L.T, dtype, DEV)
        h = L.new(L.T, 2 * F) if i % 2 else None
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h, act=ACTS[name])
        ref_h, e = L.h()
        ref, lim = glu_limits(name, ref_h, e, dtype)
        check(a[:L.T], ref, lim, f"a {K} {F}")
        assert torch.isnan(a[L.T:]).all()
        if h is not None:
            check(h, ref_h, e + half_step(dtype, ref_h), f"h {K} {F}")


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", SPLITS, ids=str)
def test_backward(m, dtype, name, kept):
    for i, (K, F) in enumerate(SIZES[dtype]):
        L = Layer(m, K, F, dtype, bias=i % 2 == 0, seed=i, lists=i % 3 == 1)
        ref_h, e = L.h()
        h = None
        if kept:
            h = torch.from_numpy(ref_h).to(dtype)
            ref_h, e = to64(h), np.zeros_like(e)
            h = h.to(DEV)
        wide = i % 2 == 1 or dtype == torch.float32
        dw0 = torch.randn(L.G, 2 * F, K, generator=torch.Generator().manual_seed(9))
        dw = dw0.to(DEV) if wide else L.new(L.G, 2 * F, K)
        dws = [t for t in dw] if i % 3 == 1 else dw
        db = L.new(L.G, 2 * F) if i % 2 == 0 else None
        dh, a = L.new(L.T, 2 * F), L.new(L.T, F) if i % 2 else None
        dx = nan_tail(L.T + 2, K, L.T, dtype, DEV)
        gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dws, L.ws, h=h, bias=L.db_, a=a, db=db, act=ACTS[name],
                           accumulate=wide)
        ref_dh, lim = grad_limits(name, ref_h, e, to64(L.da), dtype)
        check(dh, ref_dh, lim, f"dh {K} {F}")
        if a is not None:
            check(a, *glu_limits(name, ref_h, e, dtype), f"a {K} {F}")
        assert torch.isnan(dx[L.T:]).all()
        # the products of dh as it came out
        x, w, d = to64(L.x), to64(L.w), to64(dh)
        rx, rw, rb = gated.glu_backward(x, w, d, L.m)
        mx, mw, mb = gated.glu_backward(np.abs(x), np.abs(w), np.abs(d), L.m)
        n = np.array(L.m)[:, None, None]
        check(dx[:L.T], rx, (2 * F + 2) * 2 * V * mx + half_step(dtype, rx), f"dx {K} {F}")
        if wide:
            rw = rw + to64(dw0)
            mw = mw + np.abs(to64(dw0))
        check(dw, rw, (n + 3) * 2 * V * mw + half_step(torch.float32 if wide else dtype, rw), f"dw {K} {F}")
        if db is not None:
            check(db, rb, (n[..., 0] + 2) * 2 * V * mb + half_step(dtype, rb), f"db {K} {F}")


@pytest.mark.parametrize("name", ACTS)
def test_gradient_against_differences(name):
    """dx and dw of the fp32 layer against central differences of the float64 oracle."""
    L = Layer([3, 2], 8, 4, torch.float32, seed=4)
    dh, dx, dw, db = L.new(5, 8), L.new(5, 8), L.new(2, 8, 8), L.new(2, 8)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dw, L.ws, bias=L.db_, db=db, act=ACTS[name])
    x, w, b, da = (to64(t) for t in (L.x, L.w, L.b, L.da))
    loss = lambda x, w, b: float((gated.glu(name, gated.product(x, w, b, L.m)) * da).sum())  # noqa: E731
    eps = 1e-5  # error of a central difference: eps^2 / 6 times the third derivative, and 1e-16 loss / eps
    for got, which in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w, b]
        num = np.zeros_like(args[which])
        for i in np.ndindex(num.shape):
            up, dn = [t.copy() for t in args], [t.copy() for t in args]
            up[which][i] += eps
            dn[which][i] -= eps
            num[i] = (loss(*up) - loss(*dn)) / (2 * eps)
        scale = np.abs(num).max()
        check(got, num, np.full(num.shape, 2e-6 * (scale + 1)), f"gradient {which}")


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows(dtype):
    L = Layer([0, 0], 16, 8, dtype)
    a = torch.full((2, 8), float("nan"), dtype=dtype, device=DEV)
    gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_)
    assert torch.isnan(a).all()
    dw, db = L.new(2, 16, 16).fill_(7), L.new(2, 16).fill_(7)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, L.new(0, 16), L.new(0, 16), dw, L.ws, db=db)
    assert (dw == 0).all() and (db == 0).all()
    dw = torch.full((2, 16, 16), 7.0, device=DEV)
    gl.gl_glu_backward(L.dx_, L.dw_, L.dda, L.new(0, 16), None, dw, L.ws, accumulate=True)
    assert (dw == 7).all()


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T", [4, 300])
def test_infinities_and_nan(name, T):
    """A gate of +-inf takes the activation's limit, NaN stays with its row, and no other
    row is touched."""
    L = Layer([T], 16, 8, torch.float32, bias=False, seed=2)
    base = L.new(T, 8)
    gl.gl_glu_forward(L.dx_, L.dw_, base, L.ws, act=ACTS[name])
    x, w = L.dx_.clone(), L.dw_.clone()
    w[0, :8] = 0
    w[0, :8, 0] = 1  # the gate is x[:, 0]
    x[:, 0] = 0.5
    x[0, 0], x[1, 0], x[2, 0] = float("inf"), float("-inf"), float("nan")
    w[0, 8:, 0] = 0  # inf * 0 would be NaN in the other half: x[:, 0] must not reach it
    a = L.new(T, 8)
    gl.gl_glu_forward(x, w, a, L.ws, act=ACTS[name])
    assert torch.isnan(a[:3]).all()  # inf * 0 is NaN in the sum of the other half
    assert torch.isfinite(a[3:]).all()
    # kept values go straight into the activation
    h = torch.tensor([[float("inf"), 2.0], [float("-inf"), 2.0], [float("nan"), 2.0], [200.0, 2.0], [-200.0, 2.0]])
    h = h.repeat_interleave(4, 1).to(DEV)
    L5 = Layer([5], 16, 4, torch.float32, bias=False)
    da = torch.full((5, 4), 3.0, device=DEV)
    dh, dw = torch.empty(5, 8, device=DEV), torch.empty(1, 8, 16, device=DEV)
    out = torch.empty(5, 4, device=DEV)
    gl.gl_glu_backward(L5.dx_, L5.dw_, da, dh, None, dw, L5.ws, h=h, a=out, act=ACTS[name])
    assert (out[0] == float("inf")).all() and (out[1] == 0).all() and torch.isnan(out[2]).all()
    assert (out[3] == 400).all() and (out[4] == 0).all()
    assert (dh[0, :4] == 6).all() and (dh[0, 4:] == float("inf")).all()  # slope 1
    assert (dh[1] == 0).all() and torch.isnan(dh[2]).all()
    assert (dh[3, :4] == 6).all() and (dh[3, 4:] == 600).all() and (dh[4] == 0).all()


def test_nan_and_infinite_weights_stay_in_their_group():
    L = Layer([5, 20, 3], 64, 32, torch.bfloat16, seed=6)
    want = L.new(28, 32)
    gl.gl_glu_forward(L.dx_, L.dw_, want, L.ws, bias=L.db_)
    w = L.dw_.clone()
    w[1] = float("nan")
    got = L.new(28, 32)
    gl.gl_glu_forward(L.dx_, w, got, L.ws, bias=L.db_)
    assert torch.isnan(got[5:25]).all()
    assert_bits_equal(got[:5], want[:5])
    assert_bits_equal(got[25:], want[25:])


@pytest.mark.parametrize("T", [7, 700])
def test_repeats_bit_for_bit_and_dh_may_be_h(T):
    L = Layer([T - 3, 3], 128, 64, torch.bfloat16, seed=8)
    outs = []
    for _ in range(3):
        a, h = L.new(T, 64), L.new(T, 128)
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, h=h)
        dh, dx, dw = L.new(T, 128), L.new(T, 128), L.new(2, 128, 128)
        gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dw, L.ws, h=h)
        dx2, dw2 = L.new(T, 128), L.new(2, 128, 128)
        gl.gl_glu_backward(L.dx_, L.dw_, L.dda, h, dx2, dw2, L.ws, h=h)  # in place
        for p, q in ((h, dh), (dx2, dx), (dw2, dw)):
            assert_bits_equal(p, q)
        outs.append((a, dh, dx, dw))
    for o in outs[1:]:
        for p, q in zip(o, outs[0]):
            assert_bits_equal(p, q)


def test_other_stream_and_graph_replays():
    L = Layer([5, 0, 90, 33], 128, 64, torch.bfloat16, seed=3)
    T = L.T
    a, dh, dx, dw = L.new(T, 64), L.new(T, 128), L.new(T, 128), L.new(4, 128, 128)

    def step(stream=None):
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws, bias=L.db_, stream=stream)
        gl.gl_glu_backward(L.dx_, L.dw_, L.dda, dh, dx, dw, L.ws, bias=L.db_, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (a, dh, dx, dw)]
    s = torch.cuda.Stream()
    for t in (a, dh, dx, dw):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    for p, q in zip((a, dh, dx, dw), want):
        assert_bits_equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):  # new inputs in the same places, eager work in between
        L.dx_.copy_((torch.randn(T, 128, generator=torch.Generator().manual_seed(k))).to(torch.bfloat16))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (a, dh, dx, dw)]
        for t in (a, dh, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((a, dh, dx, dw), want):
            assert_bits_equal(p, q)


def test_two_calls_at_once():
    """Two streams, a workspace each: neither disturbs the other."""
    Ls = [Layer([40, 300], 256, 128, torch.bfloat16, seed=k) for k in range(2)]
    outs = [L.new(L.T, 128) for L in Ls]
    for L, o in zip(Ls, outs):
        gl.gl_glu_forward(L.dx_, L.dw_, o, L.ws, bias=L.db_)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    streams = [torch.cuda.Stream() for _ in Ls]
    for _ in range(8):
        for L, o, s in zip(Ls, outs, streams):
            gl.gl_glu_forward(L.dx_, L.dw_, o, L.ws, bias=L.db_, stream=s)
    torch.cuda.synchronize()
    for p, q in zip(outs, want):
        assert_bits_equal(p, q)


def test_invalid_splits_and_strides():
    L = Layer([5, 6], 64, 32, torch.bfloat16)
    a = L.new(11, 32).fill_(3)
    gl.gl_offsets(torch.tensor([5, 7], dtype=torch.int64, device=DEV), 11, L.ws)
    gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws)
    assert gl.gl_read_status(L.ws) == gl.GL_STATUS_SUM_MISMATCH and (a == 3).all()
    with pytest.raises(ValueError):
        gl.gl_glu_forward(L.dx_, L.dw_, L.new(32, 11).t(), L.ws)
    with pytest.raises(ValueError):
        gl.gl_glu_forward(L.new(11, 128)[:, ::2], L.dw_, a, L.ws)
    with pytest.raises(ValueError):
        gl.gl_glu_forward(L.dx_, L.dw_, a, L.ws[:64])
    with pytest.raises(ValueError):  # a group's weights off a 16-byte boundary
        flat = L.new(2 * 64 * 64 + 4)
        gl.gl_glu_forward(L.dx_, [flat[4 + 4096 * i:4 + 4096 * (i + 1)].view(64, 64) for i in range(2)], a, L.ws)
