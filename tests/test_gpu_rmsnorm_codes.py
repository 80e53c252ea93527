"""MXFP8 codes of the RMS norm: their rounding of 24-bit values, bit for bit."""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
import oracle

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
