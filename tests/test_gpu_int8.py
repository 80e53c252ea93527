"""Rows as 8-bit integers and the grouped products of 8-bit integers, plain and gated, against
the float64 oracle.  The codes and scales are equal bit for bit.  A product's sum is exact; it
is rounded to fp32, times the scales' rounded product, rounded, plus the bias, rounded:
E_h = 2^-24 (3 |sum scales| + |h|) and v^2 terms, taken as 2^-22 (|h - b| + |h|); the gated outputs go on
from there as the float layer's do."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import assert_bits_equal, nan_tail, to64
from oracle import gated
from test_gpu_glu import ACTS, TYPES, check, glu_limits, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (5, 512), (70, 1040), (9, 4096), (2, 20000), (1000, 64)])
def test_quantize(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, cols, generator=g) * torch.logspace(-6, 3, rows)[:, None]
    x[0, 3] = -0.0
    if rows > 2:
        x[1] = 0  # a row of zeros
        x[2, cols // 2] = float("inf") if cols % 32 else float("nan")
    x = x.to(dtype)
    data, scale = torch.empty(rows, cols, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    gl.gl_quantize_int8(x.to(DEV), data, scale)
    q, s = gated.quantize_int8(x.float().numpy())
    assert np.array_equal(data.cpu().numpy(), q)
    assert np.array_equal(scale.cpu().numpy(), s, equal_nan=True)


def test_quantize_every_magnitude():
    """fp32 rows from subnormals to the largest value, and ties."""
    e = np.arange(-149, 128)
    x = np.zeros((e.size, 16), np.float32)
    x[:, 0] = np.ldexp(1.0, e)
    x[:, 1:] = x[:, :1] * np.linspace(-1, 1, 15, dtype=np.float32)
    x = np.concatenate([x, np.full((1, 16), np.finfo(np.float32).max, np.float32)])
    t = torch.from_numpy(x).to(DEV)
    data, scale = torch.empty(t.shape, dtype=torch.int8, device=DEV), torch.empty(t.shape[0], device=DEV)
    gl.gl_quantize_int8(t, data, scale)
    q, s = gated.quantize_int8(x)
    assert np.array_equal(data.cpu().numpy(), q) and np.array_equal(scale.cpu().numpy(), s)


class Int8:
    def __init__(self, m, K, N, out, seed=0, bias=True, lists=False):
        g = torch.Generator().manual_seed(seed)
        G, T = len(m), int(sum(m))
        code = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int8)  # noqa: E731
        self.m, self.T, self.N, self.out = m, T, N, out
        self.x, self.w = code(T, K), code(G, N, K)
        self.xs = torch.rand(T, generator=g) * 0.02
        self.wsc = (torch.rand(G, N, generator=g) - 0.2) * K ** -0.5 * 0.02  # a scale may be negative
        self.b = torch.randn(G, N, generator=g).to(out) if bias else None
        self.ws = gl.new_workspace(G)
        gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), T, self.ws)
        dev = (lambda t: None if t is None else [v.to(DEV) for v in t]) if lists else (lambda t: None if t is None else t.to(DEV))
        self.args = (self.x.to(DEV), self.xs.to(DEV), dev(self.w), dev(self.wsc))
        self.bias = dev(self.b)

    def h(self):
        v = [None if t is None else to64(t) for t in (self.x, self.xs, self.w, self.wsc, self.b)]
        h = gated.product_int8(*v, self.m)
        return h, 2.0 ** -22 * (np.abs(gated.product_int8(*v[:4], None, self.m)) + np.abs(h))


SPLITS = [[1], [0, 2, 0], [16, 17, 1], [64, 0, 65, 5], [130, 257, 0, 40], [300]]
SIZES = [(16, 8), (48, 24), (128, 120), (208, 136), (400, 264)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("m", SPLITS, ids=str)
def test_product(m, out):
    for i, (K, N) in enumerate(SIZES):
        P = Int8(m, K, N, out, seed=i, bias=i % 2 == 0, lists=i % 3 == 1)
        y = nan_tail(P.T + 2, N, P.T, out, DEV)
        gl.gl_forward_int8(*P.args, y, P.ws, bias=P.bias)
        h, e = P.h()
        check(y[:P.T], h, e + half_step(out, h), f"y {K} {N}")
        assert torch.isnan(y[P.T:]).all()


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("m", SPLITS, ids=str)
def test_gated_product(m, out, name):
    for i, (K, F) in enumerate(SIZES):
        P = Int8(m, K, 2 * F, out, seed=i, bias=i % 2 == 0, lists=i % 3 == 1)
        a = nan_tail(P.T + 2, F, P.T, out, DEV)
        gl.gl_glu_forward_int8(*P.args, a, P.ws, bias=P.bias, act=ACTS[name])
        check(a[:P.T], *glu_limits(name, *P.h(), out), f"a {K} {F}")
        assert torch.isnan(a[P.T:]).all()


def test_sums_are_exact_at_the_longest_row():
    """All codes -128 at the longest row: 2^31 - 2^18 in int32."""
    K = (1 << 17) - 16
    x, w = (torch.full(s, -128, dtype=torch.int8, device=DEV) for s in ((3, K), (1, 8, K)))
    ws = gl.new_workspace(1)
    for T in (3,):
        gl.gl_offsets(torch.tensor([T], dtype=torch.int64, device=DEV), T, ws)
        y = torch.empty(T, 8, device=DEV)
        gl.gl_forward_int8(x, torch.ones(T, device=DEV), w, torch.ones(1, 8, device=DEV), y, ws)
        assert (y == float(K * 16384)).all()


def test_nan_scale_reaches_its_row_alone():
    P = Int8([4, 3], 64, 32, torch.bfloat16, bias=False)
    y0, y = (torch.empty(7, 32, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    gl.gl_forward_int8(*P.args, y0, P.ws)
    P.args[1][5] = float("nan")
    gl.gl_forward_int8(*P.args, y, P.ws)
    assert torch.isnan(y[5]).all()
    keep = [0, 1, 2, 3, 4, 6]
    assert_bits_equal(y[keep], y0[keep])


@pytest.mark.parametrize("T", [6, 500])
def test_mlp_in_8_bit_integers(T):
    """The run of calls of a served expert layer: rows quantized, gated product, quantized again,
    second product; against the same steps of the oracle from the codes of each step."""
    g = torch.Generator().manual_seed(T)
    G, K, F, N, bf = 3, 128, 96, 64, torch.bfloat16
    m = [T - 4, 0, 4]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w1, w2 = r(T, K).to(bf).to(DEV), (r(G, 2 * F, K) * K ** -0.5).to(bf).to(DEV), (r(G, N, F) * F ** -0.5).to(bf).to(DEV)
    new = lambda *s, dtype=torch.int8: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    f32 = torch.float32
    xq, xs = gl.gl_quantize_int8(x, new(T, K), new(T, dtype=f32))
    w1q, w1s = gl.gl_quantize_int8(w1, new(G, 2 * F, K), new(G, 2 * F, dtype=f32))
    w2q, w2s = gl.gl_quantize_int8(w2, new(G, N, F), new(G, N, dtype=f32))
    ws = gl.new_workspace(G)
    gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), T, ws)
    a, y = new(T, F, dtype=bf), new(T, N, dtype=bf)
    gl.gl_glu_forward_int8(xq, xs, w1q, w1s, a, ws)
    aq, as_ = gl.gl_quantize_int8(a, new(T, F), new(T, dtype=f32))
    gl.gl_forward_int8(aq, as_, w2q, w2s, y, ws)
    h = gated.product_int8(*(to64(t) for t in (xq, xs, w1q, w1s)), None, m)
    check(a, *glu_limits("silu", h, 2.0 ** -21 * np.abs(h), bf), "a")
    ref = gated.product_int8(*(to64(t) for t in (aq, as_, w2q, w2s)), None, m)
    check(y, ref, 2.0 ** -21 * np.abs(ref) + half_step(bf, ref), "y")
    # and near the layer in bf16: each of the three quantizations (x, a and the weights) is off by
    # at most half a step of a row's scale, 1 / 254 of its largest value
    full = new(T, F, dtype=bf)
    gl.gl_glu_forward(x, w1, full, ws)
    off = (a.float() - full.float()).norm() / full.float().norm()
    assert off < 0.05, off


def test_other_stream_and_graph_replays():
    P = Int8([5, 0, 90, 33], 128, 64, torch.bfloat16, seed=3)
    src = torch.randn(P.T, 128, device=DEV)
    y, a = torch.empty(P.T, 64, dtype=torch.bfloat16, device=DEV), torch.empty(P.T, 32, dtype=torch.bfloat16, device=DEV)

    def step(stream=None):
        gl.gl_quantize_int8(src, P.args[0], P.args[1], stream=stream)
        gl.gl_forward_int8(*P.args, y, P.ws, bias=P.bias, stream=stream)
        gl.gl_glu_forward_int8(*P.args, a, P.ws, bias=P.bias, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, a)]
    s = torch.cuda.Stream()
    y.zero_(), a.zero_()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    for p, q in zip((y, a), want):
        assert_bits_equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        src.copy_(torch.randn(P.T, 128, generator=torch.Generator().manual_seed(k)))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, a)]
        y.zero_(), a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((y, a), want):
            assert_bits_equal(p, q)


def test_strides_refused():
    P = Int8([5, 6], 64, 32, torch.bfloat16)
    y = torch.empty(11, 32, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        gl.gl_forward_int8(P.args[0].t().contiguous().t(), *P.args[1:], y, P.ws)
    with pytest.raises(ValueError):
        gl.gl_quantize_int8(torch.zeros(64, 11, device=DEV).t(), P.args[0], P.args[1])
    with pytest.raises(ValueError):
        gl.gl_forward_int8(*P.args, y, P.ws[:100])
