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


def test_routing_of_more_than_2_to_the_28_tokens():
    T, E, k = (1 << 28) + P + 3, 8, 1
    l = torch.randn(P, E, generator=torch.Generator().manual_seed(2)).to(BF16).to(DEV)
    dw = torch.randn(P, k, generator=torch.Generator().manual_seed(3)).to(DEV)

    def go(l, dw, **plan):
        ids = torch.full((l.shape[0], k), -9, dtype=torch.int32, device=DEV)
        w, dl = torch.full(ids.shape, -9.0, device=DEV), torch.full_like(l, -9)
        gl.gl_route_forward(l, ids, w, renormalize=False, **plan)
        gl.gl_route_backward(l, ids, dw, dl, renormalize=False)
        return ids, w, dl

    first = go(l, dw)
    m = torch.full((E,), -9, dtype=torch.int64, device=DEV)
    rows, slots = torch.full((T, k), -9, dtype=torch.int32, device=DEV), torch.full((T * k,), -9, dtype=torch.int32, device=DEV)
    ws = torch.empty(gl.gl_route_workspace_size(T, E), dtype=torch.uint8, device=DEV)
    got = go(repeated(l, T), repeated(dw, T), m_splits=m, row_index=rows, slot_index=slots, workspace=ws)
    ids = got[0].reshape(-1)
    assert torch.equal(ids, repeated(first[0], T).reshape(-1))
    assert repeats(got[1], first[1]) and repeats(got[2], first[2])
    assert torch.equal(m, torch.stack([(ids == e).sum() for e in range(E)]))
    assert torch.equal(slots[rows.reshape(-1).long()], torch.arange(T, dtype=torch.int32, device=DEV))
    by_row = ids[slots.long()]
    ahead, same = by_row[1:] > by_row[:-1], by_row[1:] == by_row[:-1]
    assert bool((ahead | (same & (slots[1:] > slots[:-1]))).all())


def test_routing_gradient_of_more_than_2_to_the_26_tokens_over_many_experts():
    T, E, k = (1 << 26) + P + 3, 264, 1
    l = torch.randn(P, E, generator=torch.Generator().manual_seed(4)).to(BF16).to(DEV)
    ids, w = torch.empty(P, k, dtype=torch.int32, device=DEV), torch.empty(P, k, device=DEV)
    gl.gl_route_forward(l, ids, w, renormalize=False)
    first, dw = torch.empty_like(l), w.clone()
    gl.gl_route_backward(l, ids, dw, first, renormalize=False)
    big = repeated(l, T)  # 35 GB
    out = torch.full_like(big, -9)
    gl.gl_route_backward(big, repeated(ids, T), repeated(dw, T), out, renormalize=False)
    assert torch.equal(out[:P], first)
    for t in range(0, T - P, 1 << 20):  # in parts: a comparison's own memory
        t -= t % P
        assert torch.equal(out[t:t + P], first), t
    assert torch.equal(out[T - T % P - P:T - T % P], first) and torch.equal(out[T - T % P:], first[: T % P])
