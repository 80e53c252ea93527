"""MXFP8 codes of the RMS norm: their rounding of 24-bit values, bit for bit, and their way
into the grouped forward by the routing's plan."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
import oracle
from gl_testutil import TOL_BF16, TOL_F32, assert_close, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def between_the_codes():
    """fp32 values where E4M3's rounding decides: every code, the middle of every two
    neighbours (from 0 to the first one as well), past 448 up to 512, one fp32 step to either
    side of each, and values anywhere."""
    codes = np.sort(np.abs(oracle.e4m3_decode(np.arange(127, dtype=np.uint8)))).astype(np.float32)
    at = np.concatenate([codes, (codes[1:] + codes[:-1]) / 2, np.float32([456, 464, 480, 496])])
    at = at.astype(np.float32)
    near = np.concatenate([at, np.nextafter(at, np.float32(np.inf)), np.nextafter(at, np.float32(0)), [np.nextafter(np.float32(512), np.float32(0))]])
    g = np.random.default_rng(1)
    return np.concatenate([near, np.exp2(g.uniform(-12, 9, 31 * 200 - near.size % 31)).astype(np.float32)]).astype(np.float32)


@pytest.mark.parametrize("dtype,powers", [(F32, (-40, -3, 0, 17)), (BF16, (-40, -3, 0, 17)), (F16, (-9, -3, 0, 5))])
def test_codes_round_24_bit_values_to_nearest_even(dtype, powers):
    """Rows of one magnitude 2^p with eps 0 have rstd 2^-p exactly, so y is +-gamma: its codes
    are the rule's of 24-bit values.  Each block of 32 starts with a value that fixes its scale
    (300: codes as they are), and whole blocks are moved by powers of two."""
    v = between_the_codes()
    v = np.resize(v, -(-v.size // 31) * 31).reshape(-1, 31)
    blocks = np.concatenate([np.full((len(v), 1), 300, np.float32), v], 1)
    gam = np.concatenate([blocks * np.float32(2.0 ** e) for e in (0, -30, 60, -126 - 9)])
    C = 1 << 15
    gam = np.resize(gam, (C // 32, 32)).reshape(C)
    sign = torch.randint(0, 2, (len(powers), C), generator=torch.Generator().manual_seed(2)) * 2 - 1
    x = (sign * torch.exp2(torch.tensor(powers).float())[:, None]).to(dtype)
    data = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    scale = torch.empty(len(x), C // 32, dtype=torch.uint8, device=DEV)
    gl.gl_rmsnorm_forward(x.to(DEV), torch.from_numpy(gam).to(DEV), 0.0, data=data, scale=scale)
    q, s = oracle.quantize_mxfp8(sign.numpy() * gam.astype(np.float64))
    assert np.array_equal(scale.cpu().numpy(), s)
    bad = data.cpu().numpy() != q
    assert not bad.any(), f"{int(bad.sum())} codes, first of {gam[np.argwhere(bad)[0][1]]!r}"


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("out", [BF16, F32])
def test_codes_feed_the_grouped_forward(T, out):
    """The norm's codes and scales, rows gathered into the plan's order, are gl_forward's
    MXFP8 operand, against the product of what they stand for."""
    K, N, E, k = 256, 136, 6, 2
    g = torch.Generator().manual_seed(T)
    x, gam = torch.randn(T, K, generator=g).to(BF16).to(DEV), (1 + 0.2 * torch.randn(K, generator=g)).to(DEV)
    u8 = dict(dtype=torch.uint8, device=DEV)
    data, scale = torch.empty(T, K, **u8), torch.empty(T, K // 32, **u8)
    gl.gl_rmsnorm_forward(x, gam, 1e-6, data=data, scale=scale)
    i32 = dict(dtype=torch.int32, device=DEV)
    ids, w = torch.empty(T, k, **i32), torch.empty(T, k, device=DEV)
    m, rows, slots = torch.empty(E, dtype=torch.int64, device=DEV), torch.empty(T, k, **i32), torch.empty(T * k, **i32)
    plan = torch.empty(gl.gl_route_workspace_size(T, E), **u8)
    gl.gl_route_forward(torch.randn(T, E, generator=g).to(DEV), ids, w, m_splits=m, row_index=rows, slot_index=slots, workspace=plan)
    ws = gl.new_workspace(E)
    gl.gl_offsets(m, T * k, ws)
    wq, wsc = torch.empty(E, N, K, **u8), torch.empty(E, N, K // 32, **u8)
    gl.gl_group_quantize_mxfp8((torch.randn(E, N, K, generator=g) * K ** -0.5).to(BF16).to(DEV), wq, wsc)
    token = (slots // k).long()
    xq, xs = data[token], scale[token]
    y = torch.empty(T * k, N, dtype=out, device=DEV)
    gl.gl_forward(xq, wq, y, ws, x_scale=xs, w_scale=wsc)
    assert gl.gl_read_status(ws) == 0
    c = lambda t: t.cpu().numpy()  # noqa: E731
    ref = oracle.forward_mxfp8(c(xq), c(xs), c(wq), c(wsc), None, m.tolist())
    assert_close(y, ref, TOL_BF16 if out == BF16 else TOL_F32, "forward of the norm's codes")
    # and the rows stand for the norm itself: E4M3 keeps 4 significant bits
    n = to64(x) / np.sqrt((to64(x) ** 2).mean(1, keepdims=True) + 1e-6) * to64(gam)
    deq = oracle.dequantize_mxfp8(c(xq), c(xs))
    assert np.linalg.norm(deq - n[c(token)]) < 2.0 ** -4 * np.linalg.norm(n[c(token)])
