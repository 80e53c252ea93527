"""Calls of so many rows that one launch cannot take them: rows that repeat every `P` have to
give the results of the first `P`, and those are checked elsewhere."""
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
P = 4096


def repeated(rows, T):
    """[T, ...]: the P rows over and over."""
    return rows.repeat(-(-T // P), *[1] * (rows.dim() - 1))[:T]


def repeats(t, first):
    n = t.shape[0] // P * P
    whole = bits(t[:n]).view(-1, *first.shape) == bits(first)
    return bool(whole.all()) and torch.equal(bits(t[n:]), bits(first[: t.shape[0] - n]))


def test_norm_of_more_than_2_to_the_26_rows():
    T, C = (1 << 26) + P + 3, 32
    g = torch.Generator().manual_seed(1)
    base, gam = torch.randn(P, C, generator=g).to(BF16).to(DEV), torch.randn(C, generator=g).to(BF16).to(DEV)

    def go(x):
        out = dict(h=torch.full_like(x, -1), y=torch.full_like(x, -1), data=torch.full(x.shape, 0x55, dtype=torch.uint8, device=DEV),
                   scale=torch.full((x.shape[0], C // 32), 0x55, dtype=torch.uint8, device=DEV))
        gl.gl_rmsnorm_forward(x, gam, 1e-6, residual=x, **out)
        return out

    first, all_rows = go(base), go(repeated(base, T))  # 4.3 GB a tensor
    for n in first:
        assert repeats(all_rows[n], first[n]), n
