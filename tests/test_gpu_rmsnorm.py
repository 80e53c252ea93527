"""GPU parity of the RMS norm (residual, MXFP8 output) and its backward against the
float64 oracle.

Tolerances, derived from the formulas: u is the output type's half ulp (2^-8 bf16, 2^-11
fp16 with 2^-25 below its normal range, 2^-24 fp32), e = 2^-24 an fp32 operation.
  h   one fp32 add and the rounding: (u + e) |h|
  y   sum of squares: chains of at most C / 512 + 64 adds, all terms positive, so its
      relative error is at most (C / 512 + 70) e and half of that in rstd; then the
      square root, the division, two products and the add before: (u + (C / 1024 + 48) e) |y|
  dx  the same relative errors on each term of the sum, the row mean bounded through the
      sum of its terms' magnitudes M = mean|v xh|:
      u |dx| + (C / 256 + 100) e (|dh| + rstd (|v| + |xh| M))
  dgamma  a chain of at most T / 128 + 600 adds: (T / 128 + 700) e sum|dy xh| (+ u |dgamma|)
"""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
import oracle
from gl_testutil import assert_bits_equal, bits, to64
from oracle import expert_block as eb

pytestmark = pytest.mark.gpu
DEV = "cuda"
E24 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: E24}
FLOOR = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def within(got, ref, lim, what):
    g = to64(got)
    bad = ~(np.abs(g - ref) <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside their bound; worst "
                           f"{np.max(np.where(bad, np.abs(g - ref) / (lim + 1e-300), 0)):.3g} times it")


def inputs(seed, T, C, dtype, gdtype):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return (r(T, C) * 3).to(dtype), (r(T, C) * 5).to(dtype), (1 + 0.3 * r(C)).to(gdtype), r(T, C).to(dtype), r(T, C).to(dtype)


def check_y(y, h64, ref, dtype, C, what):
    within(y, ref, (U[dtype] + (C / 1024 + 48) * E24) * np.abs(ref) + FLOOR[dtype], what)


# rows from one to many, widths of one vector, odd counts of vectors, at and past what a workgroup holds in registers
SHAPES = [(1, 8), (3, 24), (5, 72), (2, 512), (7, 520), (33, 1000), (4, 2048), (3, 4096), (2, 4104), (5, 7168), (2, 8200),
          (1, 16384), (3, 16392), (1, 65544), (601, 64), (1111, 136)]


@pytest.mark.parametrize("T,C", SHAPES)
@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_forward(T, C, dtype, gdtype):
    x, r, gam, _, _ = inputs(T * 131 + C, T, C, dtype, gdtype)
    xd, rd, gd = x.to(DEV), r.to(DEV), gam.to(DEV)
    y, h = torch.full_like(xd, float("nan")), torch.full_like(xd, float("nan"))
    gl.gl_rmsnorm_forward(xd, gd, EPS, residual=rd, h=h, y=y)
    h64, y64 = eb.rmsnorm(to64(x), to64(gam), EPS, to64(r))
    within(h, h64, (U[dtype] + E24) * np.abs(h64) + FLOOR[dtype], "h")
    check_y(y, h64, y64, dtype, C, "y")
    y2 = torch.full_like(xd, float("nan"))
    gl.gl_rmsnorm_forward(xd, gd, EPS, y=y2)
    check_y(y2, None, eb.rmsnorm(to64(x), to64(gam), EPS)[1], dtype, C, "y without residual")
    # h in place of the residual, y in place of x
    gl.gl_rmsnorm_forward(xd, gd, EPS, residual=rd, h=rd, y=xd)
    assert_bits_equal(rd, h, "h in place")
    assert_bits_equal(xd, y, "y in place")


@pytest.mark.parametrize("T,C", [(1, 32), (3, 96), (5, 544), (2, 2048), (3, 4128), (2, 8192), (1, 16416), (1, 65568), (333, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_mxfp8_output(T, C, dtype):
    """A code stands within half a step of y; the scale is the rule's except where the
    block's largest value is within the norm's own error of a power of two."""
    x, r, gam, _, _ = inputs(T * 7 + C, T, C, dtype, F32)
    data = torch.full((T, C), 0x55, dtype=torch.uint8, device=DEV)
    scale = torch.full((T, C // 32), 0x55, dtype=torch.uint8, device=DEV)
    gl.gl_rmsnorm_forward(x.to(DEV), gam.to(DEV), EPS, residual=r.to(DEV), data=data, scale=scale)
    _, y = eb.rmsnorm(to64(x), to64(gam), EPS, to64(r))
    rel = (C / 1024 + 48) * E24
    amax = np.abs(y).reshape(T, -1, 32).max(-1)
    lo, hi = (np.floor(np.log2(amax * (1 + s * rel))) - 8 + 127 for s in (-1, 1))
    s = scale.cpu().numpy().astype(np.float64)
    assert ((s == lo) | (s == hi)).all()
    step = np.repeat(np.exp2(s - 127), 32, axis=1)
    deq = oracle.dequantize_mxfp8(data.cpu().numpy(), scale.cpu().numpy())
    v = np.abs(y) / step
    half = np.maximum(np.exp2(np.floor(np.log2(np.maximum(v, 1e-300))) - 4), 2.0 ** -10)
    half = np.where(v > 448, v - 448, half)  # saturated
    bad = np.abs(deq - y) > (half * (1 + 1e-3) + 2 * rel * v) * step
    assert not bad.any(), f"{int(bad.sum())} codes further than half a step"
    # with y too: the same codes, and y as without them
    y1, y2 = (torch.empty(T, C, dtype=dtype, device=DEV) for _ in range(2))
    data2, scale2 = torch.empty_like(data), torch.empty_like(scale)
    gl.gl_rmsnorm_forward(x.to(DEV), gam.to(DEV), EPS, residual=r.to(DEV), y=y1, data=data2, scale=scale2)
    gl.gl_rmsnorm_forward(x.to(DEV), gam.to(DEV), EPS, residual=r.to(DEV), y=y2)
    assert torch.equal(data, data2) and torch.equal(scale, scale2)
    assert_bits_equal(y1, y2, "y")


def test_mxfp8_codes_are_the_quantizers_where_y_is_exact():
    """Rows of one magnitude 2^p with eps 0 have rstd 2^-p exactly, so y is +-gamma: codes
    and scales are bit for bit those of the rowwise quantizer's rule."""
    g = torch.Generator().manual_seed(5)
    T, C = 9, 1024
    gam = (torch.randn(C, generator=g) * torch.exp2(torch.randint(-90, 90, (C,), generator=g).float())).to(BF16)
    gam[:64] = 0.0
    gam[64:96] = torch.exp2(torch.arange(-133, -101).float()).to(BF16)
    sign = torch.randint(0, 2, (T, C), generator=g) * 2 - 1
    x = (sign * torch.exp2(torch.arange(T).float() * 3 - 12)[:, None]).to(BF16)
    data = torch.empty(T, C, dtype=torch.uint8, device=DEV)
    scale = torch.empty(T, C // 32, dtype=torch.uint8, device=DEV)
    y = torch.empty(T, C, dtype=BF16, device=DEV)
    gl.gl_rmsnorm_forward(x.to(DEV), gam.to(DEV), 0.0, y=y, data=data, scale=scale)
    assert_bits_equal(y, (sign.float() * gam.float()).to(BF16), "y")
    q, s = oracle.quantize_mxfp8(to64(y))
    assert np.array_equal(data.cpu().numpy(), q) and np.array_equal(scale.cpu().numpy(), s)


def test_infinities_nan_and_zeros_stay_in_their_row():
    T, C = 6, 256
    x, r, gam, _, _ = inputs(9, T, C, BF16, BF16)
    x[1, 5] = float("inf")
    x[2, 77] = float("nan")
    x[3] = 0
    r[3] = 0
    x[4] = 3e38  # its square overflows fp32
    r[4] = 0
    y = torch.empty(T, C, dtype=BF16, device=DEV)
    h = torch.empty_like(y)
    data = torch.empty(T, C, dtype=torch.uint8, device=DEV)
    scale = torch.empty(T, C // 32, dtype=torch.uint8, device=DEV)
    gl.gl_rmsnorm_forward(x.to(DEV), gam.to(DEV), EPS, residual=r.to(DEV), h=h, y=y, data=data, scale=scale)
    h64, y64 = eb.rmsnorm(to64(x), to64(gam), EPS, to64(r))
    for t in (0, 3, 5):
        check_y(y[t:t + 1], None, y64[t:t + 1], BF16, C, f"row {t}")
    q, s = oracle.quantize_mxfp8(np.zeros((1, C)))
    assert np.array_equal(data[3:4].cpu().numpy() & 0x7F, q & 0x7F) and np.array_equal(scale[3:4].cpu().numpy(), s)
    assert torch.isnan(y[1, 5]) and (y[1, :5] == 0).all() and torch.isinf(h[1, 5])
    assert torch.isnan(y[2]).all() and (scale[2] == 0xFF).all() and ((data[2] & 0x7F) == 0x7F).all()
    assert scale[1, 0] == 0xFF and (scale[1, 1:] == 0).all()
    assert (y[4] == 0).all()
    gl.gl_rmsnorm_forward(x.to(DEV), gam.to(DEV), 0.0, residual=r.to(DEV), y=y)
    assert torch.isnan(y[3]).all()  # 0 / 0, as the formula has it


def test_only_the_rows_are_written_and_no_rows_is_fine():
    x, r, gam, _, _ = inputs(10, 5, 520, BF16, BF16)
    buf = torch.full((9, 520), float("nan"), dtype=BF16, device=DEV)
    gl.gl_rmsnorm_forward(x.to(DEV), gam.to(DEV), EPS, y=buf[2:7])
    assert torch.isnan(buf[:2]).all() and torch.isnan(buf[7:]).all() and not torch.isnan(buf[2:7]).any()
    gl.gl_rmsnorm_forward(x[:0].to(DEV), gam.to(DEV), EPS, y=buf[:0])
    dg = torch.full((520,), 7.0, device=DEV)
    ws = torch.empty(gl.gl_rmsnorm_workspace_size(0, 520), dtype=torch.uint8, device=DEV)
    gl.gl_rmsnorm_backward(x[:0].to(DEV), x[:0].to(DEV), gam.to(DEV), EPS, buf[:0], dgamma=dg, accumulate=True, workspace=ws)
    assert (dg == 7).all()
    gl.gl_rmsnorm_backward(x[:0].to(DEV), x[:0].to(DEV), gam.to(DEV), EPS, buf[:0], dgamma=dg, workspace=ws)
    assert (dg == 0).all()


def test_offsets_past_32_bits():
    """More than 2^32 elements: the last rows against the oracle, forward and backward."""
    T, C = 70001, 65536
    x = torch.zeros(T, C, dtype=BF16, device=DEV)  # 9.2 GB
    g = torch.Generator().manual_seed(3)
    last, gam, dy = torch.randn(2, C, generator=g).to(BF16), torch.randn(C, generator=g).to(BF16), torch.randn(2, C, generator=g).to(BF16)
    x[-2:] = last.to(DEV)
    y = torch.empty_like(x)
    data = torch.empty(T, C, dtype=torch.uint8, device=DEV)
    scale = torch.empty(T, C // 32, dtype=torch.uint8, device=DEV)
    gl.gl_rmsnorm_forward(x, gam.to(DEV), EPS, y=y, data=data, scale=scale)
    ref = eb.rmsnorm(to64(last), to64(gam), EPS)[1]
    check_y(y[-2:], None, ref, BF16, C, "last rows")
    assert (y[:-2] == 0).all() and not (data[:-2] & 0x7F).any()
    deq = oracle.dequantize_mxfp8(data[-2:].cpu().numpy(), scale[-2:].cpu().numpy())
    assert np.linalg.norm(deq - ref) < 2.0 ** -4 * np.linalg.norm(ref)
    del data, scale
    y.zero_()
    y[-2:] = dy.to(DEV)
    dg = torch.empty(C, device=DEV)
    ws = torch.empty(gl.gl_rmsnorm_workspace_size(T, C), dtype=torch.uint8, device=DEV)
    gl.gl_rmsnorm_backward(y, x, gam.to(DEV), EPS, y, dgamma=dg, workspace=ws)  # in place of dy
    dx64, dg64 = eb.rmsnorm_backward(to64(dy), to64(last), to64(gam), EPS)
    assert (y[:-2] == 0).all()
    assert np.linalg.norm(to64(y[-2:]) - dx64) < 2.0 ** -8 * np.linalg.norm(dx64)
    assert np.linalg.norm(to64(dg) - dg64) < 1e-5 * np.linalg.norm(dg64)


def check_backward(T, C, dtype, gdtype, with_dh):
    _, h, gam, dy, dh = inputs(T * 17 + C, T, C, dtype, gdtype)
    ws = torch.empty(gl.gl_rmsnorm_workspace_size(T, C), dtype=torch.uint8, device=DEV)
    dx = torch.full((T, C), float("nan"), dtype=dtype, device=DEV)
    dg = torch.full((C,), float("nan"), device=DEV)
    args = dy.to(DEV), h.to(DEV), gam.to(DEV), EPS
    gl.gl_rmsnorm_backward(*args, dx, dh=dh.to(DEV) if with_dh else None, dgamma=dg, workspace=ws)
    H, G, DY, DH = to64(h), to64(gam), to64(dy), to64(dh) if with_dh else np.zeros((T, C))
    dx64, dg64 = eb.rmsnorm_backward(DY, H, G, EPS, DH)
    rstd = 1 / np.sqrt((H * H).mean(1, keepdims=True) + EPS)
    v, xh = np.abs(DY * G), np.abs(H * rstd)
    mag = np.abs(DH) + rstd * (v + xh * (v * xh).mean(1, keepdims=True))
    within(dx, dx64, U[dtype] * np.abs(dx64) + (C / 256 + 100) * E24 * mag + FLOOR[dtype], "dx")
    gmag = (T / 128 + 700) * E24 * (np.abs(DY) * xh).sum(0)
    within(dg, dg64, gmag, "dgamma")
    # without dgamma, in place of dy; dgamma again: the same bits, added into, in the layer's type
    dy2 = args[0].clone()
    gl.gl_rmsnorm_backward(dy2, *args[1:], dy2, dh=dh.to(DEV) if with_dh else None)
    assert_bits_equal(dy2, dx, "dx in place of dy, without dgamma")
    ws.fill_(0xFF)
    dg2 = torch.full((C,), 3.0, device=DEV)
    gl.gl_rmsnorm_backward(*args, dx, dgamma=dg2, accumulate=True, workspace=ws)
    assert torch.equal(dg2, 3.0 + dg)
    if dtype != F32:
        dgl = torch.empty(C, dtype=dtype, device=DEV)
        gl.gl_rmsnorm_backward(*args, dx, dgamma=dgl, workspace=ws)
        assert_bits_equal(dgl, dg.to(dtype), "dgamma in the layer's type")


@pytest.mark.parametrize("T,C", SHAPES)
@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)])
def test_backward(T, C, dtype, gdtype):
    check_backward(T, C, dtype, gdtype, with_dh=(T + C) % 16 != 0)


@pytest.mark.parametrize("T", [511, 512, 513, 1025, 2500])
def test_backward_rows_around_the_grid(T):
    check_backward(T, 200, BF16, F32, True)


def test_backward_against_differences():
    """dx and dgamma in fp32 against central differences of the oracle's forward in
    float64: the step's own error is about 1e-9, so fp32's bounds decide."""
    T, C = 3, 40
    _, h, gam, dy, dh = inputs(77, T, C, F32, F32)
    ws = torch.empty(gl.gl_rmsnorm_workspace_size(T, C), dtype=torch.uint8, device=DEV)
    dx, dg = torch.empty(T, C, device=DEV), torch.empty(C, device=DEV)
    gl.gl_rmsnorm_backward(dy.to(DEV), h.to(DEV), gam.to(DEV), EPS, dx, dh=dh.to(DEV), dgamma=dg, workspace=ws)
    H, G, DY, DH = (to64(t) for t in (h, gam, dy, dh))
    loss = lambda a, g: (eb.rmsnorm(a, g, EPS)[1] * DY).sum() + (a * DH).sum()  # noqa: E731
    step = 1e-5
    for t, c in ((0, 0), (1, 17), (2, 39)):
        d = np.zeros((T, C))
        d[t, c] = step
        num = (loss(H + d, G) - loss(H - d, G)) / (2 * step)
        assert abs(float(dx[t, c]) - num) < 1e-4 * (1 + abs(num))
    for c in (0, 21, 39):
        d = np.zeros(C)
        d[c] = step
        assert abs(float(dg[c]) - (loss(H, G + d) - loss(H, G - d)) / (2 * step)) < 1e-4 * (1 + abs(float(dg[c])))


def test_other_stream_and_graph_replay():
    x, r, gam, dy, _ = inputs(21, 40, 1024, BF16, BF16)
    xd, rd, gd, dyd = x.to(DEV), r.to(DEV), gam.to(DEV), dy.to(DEV)
    mk = lambda: (torch.empty_like(xd), torch.empty_like(xd), torch.empty_like(xd), torch.empty(1024, device=DEV))  # noqa: E731
    ws = torch.empty(gl.gl_rmsnorm_workspace_size(40, 1024), dtype=torch.uint8, device=DEV)

    def go(h, y, dx, dg, stream=None):
        gl.gl_rmsnorm_forward(xd, gd, EPS, residual=rd, h=h, y=y, stream=stream)
        gl.gl_rmsnorm_backward(dyd, h, gd, EPS, dx, dgamma=dg, workspace=ws, stream=stream)

    ref = mk()
    go(*ref)
    torch.cuda.synchronize()
    side, out = torch.cuda.Stream(), mk()
    side.wait_stream(torch.cuda.current_stream())
    go(*out, stream=side)
    side.synchronize()
    for a, b in zip(ref, out):
        assert_bits_equal(a, b, "other stream")
    graph, rep = torch.cuda.CUDAGraph(), mk()
    with torch.cuda.graph(graph):
        go(*rep)
    for i in range(3):
        for t in rep:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, rep):
            assert_bits_equal(a, b, f"replay {i}")
    assert bits(ref[0]).numel()
