"""GPU parity of the token routing, its plan and its gradient against the float64 oracle.

ids, m_splits and the maps are equal.  Weights, with e = 2^-24 and d the distance of a
chosen logit from the largest: the exponential's argument carries an error of e d, so the
score's relative error is at most (d + 4) e, its sum's (E / 64 + 10) e more (positive
terms): (2 D + E / 64 + 24) e relative, D the largest distance that is not masked.  The
gradient multiplies such scores into sums over the slots of |dw| w, so its bound is that
many e of the terms' magnitudes, plus the output type's rounding.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
from gl_testutil import assert_bits_equal, to64
from oracle import expert_block as eb

pytestmark = pytest.mark.gpu
DEV = "cuda"
E24 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: E24}
FLOOR = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")
SCORE = {False: gl.GL_SCORE_SOFTMAX, True: gl.GL_SCORE_SIGMOID}


def logits_of(seed, T, E, dtype, masked):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * 2).to(dtype)  # 16-bit logits tie often
    if masked:
        u = torch.rand(T, E + 1, generator=g)
        l = l.masked_fill((u[:, 1:] < 0.3) | (u[:, :1] < 0.15), -INF)
        l[u[:, 1:] > 0.97] = float("nan")
    return l


def forward(l, k, sigmoid, renorm, plan=True):
    T, E = l.shape
    out = dict(ids=torch.full((T, k), -9, dtype=torch.int32, device=DEV), weights=torch.full((T, k), float("nan"), device=DEV))
    kw = {}
    if plan:
        kw = dict(m_splits=torch.full((E,), -9, dtype=torch.int64, device=DEV),
                  row_index=torch.full((T, k), -9, dtype=torch.int32, device=DEV),
                  slot_index=torch.full((T * k,), -9, dtype=torch.int32, device=DEV))
        ws = torch.full((gl.gl_route_workspace_size(T, E),), 0xAB, dtype=torch.uint8, device=DEV)
        gl.gl_route_forward(l, out["ids"], out["weights"], score=SCORE[sigmoid], renormalize=renorm, workspace=ws, **kw)
    else:
        gl.gl_route_forward(l, out["ids"], out["weights"], score=SCORE[sigmoid], renormalize=renorm)
    return {**out, **kw}


def spread(L):
    l = np.where(np.isfinite(L), L, np.nan)
    with np.errstate(all="ignore"):
        return float(np.nan_to_num(np.nanmax(l) - np.nanmin(l))) if np.isfinite(L).any() else 0.0


def check(l, k, sigmoid, renorm):
    T, E = l.shape
    got, L = forward(l.to(DEV), k, sigmoid, renorm), to64(l)
    ids, w = eb.route(L, k, sigmoid, renorm)
    assert np.array_equal(got["ids"].cpu().numpy(), ids), "ids"
    tol = (2 * spread(L) + np.nanmax(np.abs(np.where(np.isfinite(L), L, 0))) + E / 64 + 24) * E24
    assert (np.abs(to64(got["weights"]) - w) <= tol * w + 2.0 ** -126).all(), "weights"
    splits, rows, slots = eb.plan(ids, E)
    for n, ref in (("m_splits", splits), ("row_index", rows), ("slot_index", slots)):
        assert np.array_equal(got[n].cpu().numpy(), ref), n
    alone = forward(l.to(DEV), k, sigmoid, renorm, plan=False)
    assert torch.equal(alone["ids"], got["ids"]) and torch.equal(alone["weights"], got["weights"])
    return ids


SIZES = [(1, 1, 1), (1, 7, 3), (2, 64, 8), (5, 65, 4), (63, 16, 2), (64, 8, 8), (65, 33, 5), (130, 128, 6), (257, 60, 4),
         (40, 200, 22), (17, 256, 8), (9, 1000, 32), (3, 1024, 32), (700, 5, 2)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("masked", [False, True])
def test_forward_and_plan(T, E, k, dtype, masked):
    for sigmoid in (False, True):
        for renorm in (False, True):
            check(logits_of(T * 11 + E, T, E, dtype, masked), k, sigmoid, renorm)


def test_ties_masks_and_infinities():
    low = float(torch.finfo(F32).min)
    rows = [[0.0] * 70, [-0.0, 0.0] * 35, [-INF] * 70, [float("nan")] * 70, [low] * 70, [INF] + [0.0] * 68 + [INF],
            [-INF] * 69 + [1.0], [low] * 69 + [-INF], [1e30, -1e30] * 35, [-200.0] * 69 + [200.0]]
    l = torch.tensor(rows)
    for sigmoid in (False, True):
        for renorm in (False, True):
            got = forward(l.to(DEV), 6, sigmoid, renorm)
            ids, w = eb.route(to64(l), 6, sigmoid, renorm)
            assert np.array_equal(got["ids"].cpu().numpy(), ids)
            assert np.allclose(to64(got["weights"]), w, rtol=100 * E24 * 200, atol=1e-30)
            assert (got["weights"][2:4] == 0).all()


def test_many_tokens_match_a_stable_sort():
    """Sizes past one scan: the whole plan against torch's stable sort."""
    for T, E, k in ((5000, 256, 8), (20011, 31, 3), (4097, 512, 4)):
        l = logits_of(T, T, E, BF16, True).to(DEV)
        got = forward(l, k, False, True)
        key = torch.where(torch.isnan(l), -INF, l.float())
        ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
        flat = ids.reshape(-1)
        slots = torch.sort(flat, stable=True)[1]
        assert torch.equal(got["ids"].long(), ids) and torch.equal(got["slot_index"].long(), slots)
        assert torch.equal(got["row_index"].reshape(-1)[slots].long(), torch.arange(T * k, device=DEV))
        assert torch.equal(got["m_splits"], torch.bincount(flat, minlength=E))


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens' gates, the counts, and the gradient's last rows."""
    T, E = 2200003, 1000
    l = torch.zeros(T, E, dtype=BF16, device=DEV)  # 4.4 GB
    tail = logits_of(6, 70, E, BF16, False)
    l[-70:] = tail.to(DEV)
    got = forward(l, 2, False, False)
    ids, w = eb.route(to64(tail), 2, False, False)
    assert np.array_equal(got["ids"][-70:].cpu().numpy(), ids)
    assert np.allclose(to64(got["weights"][-70:]), w, rtol=1e-5)
    counts = torch.bincount(got["ids"].reshape(-1).long(), minlength=E)
    assert torch.equal(got["m_splits"], counts) and counts[0] >= T - 70
    assert torch.equal(got["slot_index"][got["row_index"].reshape(-1).long()].long(), torch.arange(2 * T, device=DEV))
    dl = torch.empty_like(l)
    dw = torch.ones(T, 2, device=DEV)
    dw[:, 1] = -2
    gl.gl_route_backward(l, got["ids"], dw, dl, renormalize=False)
    ref = eb.route_backward(to64(tail), ids, np.tile([1.0, -2.0], (70, 1)), False, False)
    assert np.linalg.norm(to64(dl[-70:]) - ref) < 2.0 ** -8 * np.linalg.norm(ref)


def test_plan_feeds_the_offsets():
    l = logits_of(4, 300, 12, F32, False).to(DEV)
    got = forward(l, 3, False, True)
    ws = gl.new_workspace(12)
    gl.gl_offsets(got["m_splits"], 900, ws)
    assert gl.gl_read_status(ws) == 0
    off = gl.workspace_offsets(ws, 12)
    expert_of_row = got["ids"].reshape(-1)[got["slot_index"].long()]
    assert torch.equal(torch.searchsorted(expert_of_row.long(), torch.arange(13, device=DEV)), off)


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("masked", [False, True])
def test_backward(T, E, k, dtype, masked):
    l = logits_of(T * 5 + E, T, E, dtype, masked)
    L = to64(l)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T + E))
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids, w = eb.route(L, k, sigmoid, renorm)
            out = torch.full((T, E), float("nan"), dtype=dtype, device=DEV)
            gl.gl_route_backward(l.to(DEV), torch.from_numpy(ids).int().to(DEV), dw.to(DEV), out, score=SCORE[sigmoid],
                                 renormalize=renorm)
            ref = eb.route_backward(L, ids, dw.numpy(), sigmoid, renorm)
            n = (4 * spread(L) + 2 * np.nanmax(np.abs(np.where(np.isfinite(L), L, 0))) + E / 16 + 100) * E24
            mean = (np.abs(dw.numpy()) * w).sum(1, keepdims=True)
            mag = np.zeros((T, E))
            np.put_along_axis(mag, ids, w * (np.abs(dw.numpy()) + mean), 1)
            if not sigmoid and not renorm:  # every expert's share of the softmax
                full = np.zeros((T, E))
                fi, fw = eb.route(L, E, False, False)
                np.put_along_axis(full, fi, fw, 1)
                mag = np.maximum(mag, full * mean)
            bad = ~(np.abs(to64(out) - ref) <= U[dtype] * np.abs(ref) + n * mag + FLOOR[dtype])
            assert not bad.any(), f"{int(bad.sum())} of {bad.size}, sigmoid {sigmoid}, renorm {renorm}"


def test_backward_against_differences():
    """fp32 gradients against central differences of the oracle's weights in float64."""
    T, E, k, step = 6, 12, 3, 1e-6
    l = logits_of(8, T, E, F32, False)
    L, dw = to64(l), np.random.default_rng(1).normal(0, 1, (T, k))
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids, _ = eb.route(L, k, sigmoid, renorm)
            out = torch.empty(T, E, device=DEV)
            gl.gl_route_backward(l.to(DEV), torch.from_numpy(ids).int().to(DEV), torch.from_numpy(dw).float().to(DEV), out,
                                 score=SCORE[sigmoid], renormalize=renorm)
            for t in range(T):
                for e in (int(ids[t, 0]), int(ids[t, k - 1]), t):
                    d = np.zeros((T, E))
                    d[t, e] = step
                    up, down = eb.route(L + d, k, sigmoid, renorm), eb.route(L - d, k, sigmoid, renorm)
                    assert np.array_equal(up[0], ids) and np.array_equal(down[0], ids)
                    assert abs(float(out[t, e]) - ((up[1] - down[1]) * dw).sum() / (2 * step)) < 1e-5


def test_backward_of_foreign_ids_and_empty_calls():
    l = logits_of(2, 4, 10, F32, False)
    ids = torch.tensor([[1, -1], [10, 3], [-5, 99], [0, 9]], dtype=torch.int32)
    out = torch.full((4, 10), float("nan"), device=DEV)
    gl.gl_route_backward(l.to(DEV), ids.to(DEV), torch.ones(4, 2, device=DEV), out, score=gl.GL_SCORE_SIGMOID, renormalize=False)
    s = torch.sigmoid(l)
    ref = torch.zeros(4, 10)
    for t, e in ((0, 1), (1, 3), (3, 0), (3, 9)):
        ref[t, e] = s[t, e] * (1 - s[t, e])
    assert torch.allclose(out.cpu(), ref, rtol=1e-5, atol=1e-7)
    splits = torch.full((10,), -9, dtype=torch.int64, device=DEV)
    none = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    ws = torch.empty(gl.gl_route_workspace_size(0, 10), dtype=torch.uint8, device=DEV)
    gl.gl_route_forward(l[:0].to(DEV), none, none.float(), m_splits=splits, row_index=none, slot_index=none.reshape(-1), workspace=ws)
    assert (splits == 0).all()
    gl.gl_route_backward(l[:0].to(DEV), none, none.float(), out[:0])


def test_other_stream_and_graph_replay():
    l = logits_of(3, 200, 64, F32, True).to(DEV)
    ref = forward(l, 4, False, True)
    torch.cuda.synchronize()
    out = {n: torch.empty_like(t) for n, t in ref.items()}
    ws = torch.empty(gl.gl_route_workspace_size(200, 64), dtype=torch.uint8, device=DEV)
    dw, dl, dl2 = torch.ones(200, 4, device=DEV), torch.empty_like(l), torch.empty_like(l)
    gl.gl_route_backward(l, ref["ids"], dw, dl)

    def go(stream=None):
        gl.gl_route_forward(l, out["ids"], out["weights"], m_splits=out["m_splits"], row_index=out["row_index"],
                            slot_index=out["slot_index"], workspace=ws, stream=stream)
        gl.gl_route_backward(l, out["ids"], dw, dl2, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    assert all(torch.equal(ref[n], out[n]) for n in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for i in range(3):
        for t in out.values():
            t.fill_(-3)
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref[n], out[n]) for n in ref), i
        assert_bits_equal(dl, dl2, "dlogits")
