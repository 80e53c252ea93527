"""GPU parity of the expert layer for a few tokens against the float64 oracle.

Tolerance, derived: with e = 2^-24, products of 16-bit values are exact in fp32 and a sum
of n terms in any order is within n e of the terms' magnitudes.  So
  |dh| <= (K + 8) e (|W1| |x| + |b1|)
  |da| <= 1.1 |u| |dg| + |silu(g)| |du| + (32 + |g|) e |a| + 2^-16 |a|
the last term the two 16-bit parts that a is kept in for 16-bit products (fp16: 2^-24
more, the end of its range); silu's slope is below 1.1 and its exponential's argument
carries an error of e |g|.  Then
  |dy| <= sum_j w_j (|W2| |da| + (F + 16) e (|W2| |a| + |b2|)) + 64 e (...) + u |y|.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_gl_amd as gl
import oracle
from gl_testutil import assert_bits_equal, to64
from oracle import expert_block as eb

pytestmark = pytest.mark.gpu
DEV = "cuda"
E24 = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: E24}


def case(seed, T, E, k, K, F, N, dtype, mx=False, bias=False, residual=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype)  # noqa: E731
    c = dict(x=r(T, K), w1=r(E, 2 * F, K, std=K ** -0.5), w2=r(E, N, F, std=F ** -0.5), b1=r(E, 2 * F) if bias else None,
             b2=r(E, N) if bias else None, residual=r(T, N) if residual else None)
    l = torch.randn(T, E, generator=g)
    w, ids = torch.topk(torch.softmax(l, 1), min(k, E), dim=1)
    c["ids"], c["weights"] = ids.int().contiguous(), w.contiguous()
    if mx:
        for n in ("w1", "w2"):
            q = [oracle.quantize_mxfp8(to64(c[n][e])) for e in range(E)]
            c[n + "_scale"] = torch.from_numpy(np.stack([s for _, s in q]))
            c[n] = torch.from_numpy(np.stack([d for d, _ in q]))
    return c


def dense(c, n):
    if n + "_scale" not in c:
        return to64(c[n])
    return np.stack([oracle.dequantize_mxfp8(d.numpy(), s.numpy()) for d, s in zip(c[n], c[n + "_scale"])])


def run(c, y=None, stream=None, **over):
    d = {n: t.to(DEV) for n, t in c.items() if t is not None}
    d.update(over)
    T, k = c["ids"].shape
    N = d["w2"][0].shape[0]
    E, F = len(d["w2"]), d["w2"][0].shape[1]
    size = gl.gl_moe_few_tokens_workspace_size(T, k, E, F)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN wherever something is read before it is written
    if y is None:
        y = torch.full((T, N), float("nan"), dtype=c["x"].dtype, device=DEV)
    gl.gl_moe_few_tokens(d.pop("x"), d.pop("ids"), d.pop("weights"), d.pop("w1"), d.pop("w2"), y, ws, stream=stream, **d)
    return y


def bound(c):
    """(reference, limit) of every output."""
    x, ids, w, w1, w2 = to64(c["x"]), c["ids"].numpy(), to64(c["weights"]), dense(c, "w1"), dense(c, "w2")
    E, F2, K = w1.shape
    F, dtype = F2 // 2, c["x"].dtype
    b1, b2 = (None if c[n] is None else to64(c[n]) for n in ("b1", "b2"))
    res = None if c["residual"] is None else to64(c["residual"])
    ref = eb.moe(x, ids, w, w1, w2, b1, b2, res)
    lim = np.zeros_like(ref) if res is None else 64 * E24 * np.abs(res)
    for t in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if e < 0 or e >= E or w[t, j] == 0:
                continue
            h = w1[e] @ x[t] + (0 if b1 is None else b1[e])
            dh = (K + 8) * E24 * (np.abs(w1[e]) @ np.abs(x[t]) + (0 if b1 is None else np.abs(b1[e])))
            g, u = h[:F], h[F:]
            a = np.abs(oracle.silu(g) * u)
            da = 1.1 * (np.abs(u) + dh[F:]) * dh[:F] + np.abs(oracle.silu(g)) * dh[F:] + (32 + np.abs(g)) * E24 * a
            if dtype != F32:
                da = da + 2.0 ** -16 * a + (2.0 ** -24 if dtype == F16 else 0)
            mag = np.abs(w2[e]) @ a + (0 if b2 is None else np.abs(b2[e]))
            lim[t] += w[t, j] * (np.abs(w2[e]) @ da + (F + 16 + 64) * E24 * mag)
    return ref, lim + U[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == F16 else 0)


def check(c, y):
    ref, lim = bound(c)
    bad = ~(np.abs(to64(y) - ref) <= lim)
    worst = float(np.max(np.abs(to64(y) - ref) / (lim + 1e-300)))
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside their bound, worst {worst:.3g} times it"


# (T, E, k, K, F, N): one token to the most, fewer and more slots than experts, ragged widths
SIZES = [(1, 1, 1, 8, 8, 8), (1, 16, 4, 64, 32, 64), (2, 3, 2, 72, 40, 24), (5, 8, 2, 256, 136, 264), (15, 40, 3, 128, 64, 128),
         (16, 4, 2, 200, 72, 96), (17, 6, 3, 136, 48, 80), (31, 64, 8, 96, 104, 112), (33, 2, 1, 520, 16, 40),
         (48, 5, 5, 64, 88, 72), (64, 3, 2, 160, 56, 48), (64, 100, 6, 72, 24, 32), (7, 300, 30, 40, 32, 56),
         (3, 4, 2, 1032, 520, 1000)]


@pytest.mark.parametrize("T,E,k,K,F,N", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_forward(T, E, k, K, F, N, dtype):
    c = case(T * 3 + E, T, E, k, K, F, N, dtype, bias=E % 2 == 0, residual=T % 2 == 1)
    check(c, run(c))


# outputs of 4096 and more (another workgroup shape), contractions over several blocks
WIDE = [(1, 5, 3, 2600, 1112, 4104), (2, 4, 2, 1544, 520, 4096), (4, 6, 2, 1032, 200, 4104), (9, 5, 2, 520, 1096, 4200),
        (16, 3, 2, 264, 72, 4096), (24, 6, 2, 136, 264, 4104), (64, 9, 3, 72, 136, 4096)]


@pytest.mark.parametrize("T,E,k,K,F,N", WIDE)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_forward_wide(T, E, k, K, F, N, dtype):
    c = case(T * 5 + E, T, E, k, K, F, N, dtype, bias=T % 2 == 0, residual=T % 3 == 1)
    check(c, run(c))


@pytest.mark.parametrize("T,E,k,K,F,N", [(1, 5, 3, 2080, 1120, 4104), (2, 4, 2, 1056, 2176, 4096), (4, 6, 2, 1152, 224, 4104),
                                         (9, 5, 2, 544, 1088, 4200), (40, 6, 2, 128, 256, 4104),
                                         (1, 5, 3, 2048, 1152, 4104), (2, 4, 2, 1280, 2048, 80), (5, 9, 2, 512, 1152, 4104),
                                         (12, 3, 2, 384, 128, 72), (30, 4, 2, 1152, 384, 4096), (64, 3, 3, 256, 128, 40)])
def test_mxfp8_weights_wide(T, E, k, K, F, N):
    c = case(T * 7 + E, T, E, k, K, F, N, BF16, mx=True, bias=T % 2 == 0, residual=T % 3 == 1)
    check(c, run(c))


@pytest.mark.parametrize("T,E,k,K,F,N", [(1, 4, 2, 32, 32, 8), (3, 8, 2, 96, 64, 40), (5, 40, 4, 160, 96, 136),
                                         (17, 6, 3, 544, 32, 64), (40, 3, 2, 64, 288, 72), (64, 20, 4, 128, 160, 96)])
def test_mxfp8_weights(T, E, k, K, F, N):
    c = case(T + E, T, E, k, K, F, N, BF16, mx=True, bias=T % 2 == 0, residual=T % 2 == 1)
    check(c, run(c))


# rows of an odd number of 128 codes, whose last scales lie at the end of the tensor
@pytest.mark.parametrize("T,E,k,K,F,N", [(6, 2, 2, 384, 384, 40), (12, 3, 2, 640, 1152, 4104), (25, 3, 2, 1152, 640, 72),
                                         (40, 4, 3, 896, 384, 4096), (64, 3, 2, 384, 896, 24), (9, 1, 1, 256, 256, 16)])
def test_mxfp8_rows_of_odd_length(T, E, k, K, F, N):
    c = case(T * 11 + E, T, E, k, K, F, N, BF16, mx=True, bias=T % 2 == 1, residual=T % 2 == 0)
    check(c, run(c))
    c["w2_scale"][0, 1, -1] = 0xFF  # reaches column 1 of the tokens that name expert 0
    ids, w = c["ids"].cpu().numpy(), c["weights"].cpu().numpy()
    hit = torch.from_numpy(((ids == 0) & (w != 0)).any(1))
    assert torch.equal(torch.isnan(run(c)).cpu().any(1), hit) and hit.any()


def test_mxfp8_scales_at_the_ends_of_their_range():
    """Scales 2^-127 .. 2^127 and the NaN scale: codes expand exactly or to NaN."""
    c = case(5, 2, 2, 1, 64, 32, 16, BF16, mx=True)
    c["ids"] = torch.tensor([[0], [1]], dtype=torch.int32)
    c["weights"] = torch.ones(2, 1)
    c["w2_scale"][0] = 0  # 2^-127: the products vanish next to nothing else
    y = run(c)
    ref = eb.moe(to64(c["x"]), c["ids"].numpy(), to64(c["weights"]), dense(c, "w1"), dense(c, "w2"))
    assert np.abs(ref[0]).max() < 1e-35 and y[0].abs().max() < 1e-35
    c["w2_scale"][1, 3] = 0xFF
    y = run(c)
    assert torch.isnan(y[1, 3]) and not torch.isnan(y[1, :3]).any() and not torch.isnan(y[1, 4:]).any()


@pytest.mark.parametrize("F", [32, 128])
def test_mxfp8_weights_expand_exactly(F):
    """Every code under scales over their range, read off one at a time: token t has a = 2^m
    in column t of a and zeros elsewhere (g = 64 makes silu(g) = g), so y is code * scale *
    2^m, exact in bf16; a weight below 2^-126, bf16's smallest normal value, may lose bits
    there or count as 0: it is within its own size; one of 2^128 or more is infinite (times
    the zeros of the one-hot row NaN), as in fp32."""
    T, K = 32, 32
    scales = torch.tensor([0, 1, 2, 60, 126, 127, 128, 200, 253, 254], dtype=torch.uint8)
    w1 = torch.zeros(10, 2 * F, K, dtype=BF16)
    x = torch.eye(T, K).to(BF16)
    for e, s in enumerate(scales.tolist()):
        m = max(-100, min(100, 127 - s))
        for t in range(T):
            w1[e, t, t] = 64.0
            w1[e, F + t, t] = 2.0 ** (m - 6)
    q = [oracle.quantize_mxfp8(to64(w1[e])) for e in range(10)]
    w2 = torch.arange(256, dtype=torch.uint8).view(1, 256, 1).expand(10, 256, F).contiguous()
    c = dict(x=x, w1=torch.from_numpy(np.stack([d for d, _ in q])), w1_scale=torch.from_numpy(np.stack([d for _, d in q])),
             w2=w2, w2_scale=scales.view(10, 1, 1).expand(10, 256, F // 32).contiguous(), b1=None, b2=None, residual=None,
             weights=torch.ones(T, 1))
    for e, s in enumerate(scales.tolist()):
        c["ids"] = torch.full((T, 1), e, dtype=torch.int32)
        y = to64(run(c))
        m = max(-100, min(100, 127 - s))
        ref = oracle.e4m3_decode(np.arange(256, dtype=np.uint8)) * 2.0 ** (s - 127 + m)
        small = np.abs(ref) < 2.0 ** (m - 126)
        ref = np.where(small[None] & (np.abs(y - ref) <= np.abs(ref)), y, ref)
        large = np.broadcast_to(np.abs(ref) >= 2.0 ** (m + 128), y.shape)
        assert not np.isfinite(y[large]).any()
        assert np.array_equal(y[~large], ref[~large], equal_nan=True), s


@pytest.mark.parametrize("mx", [False, True])
def test_per_expert_lists_match_stacked(mx):
    c = case(11, 9, 5, 2, 96, 64, 72, BF16, mx=mx, bias=True, residual=True)
    y = run(c)
    names = ["w1", "w2", "b1", "b2"] + (["w1_scale", "w2_scale"] if mx else [])
    lists = {n: [t.to(DEV).clone() for t in c[n]] for n in names}
    assert_bits_equal(run(c, **lists), y, "lists")
    check(c, y)


@pytest.mark.parametrize("T", [1, 5, 20, 64])
def test_slots_that_take_no_part(T):
    """Ids outside the experts, weights of 0 (also where the row would give NaN) and a
    token without any slot; rows past T keep their bits; the residual in place."""
    E, k, N = 6, 3, 72
    c = case(21, T, E, k, 64, 40, N, BF16, residual=True)
    c["ids"][0] = torch.tensor([-1, E, 1 << 30])
    if T > 1:
        c["ids"][1, 1] = -7
        c["weights"][2, 0] = 0.0
        c["weights"][3] = 0.0
        c["x"][3, 5] = float("nan")
    c["w1"][E - 1, 0, 0] = float("inf")
    c["ids"][c["ids"] == E - 1] = -1  # nothing names the expert that would give NaN
    buf = torch.full((T + 4, N), 5.0, dtype=BF16, device=DEV)
    buf[:T] = c["residual"].to(DEV)
    run(c, y=buf, residual=buf[:T])
    assert (buf[T:] == 5).all()
    assert torch.equal(buf[0].cpu(), c["residual"][0])
    if T > 1:
        assert torch.equal(buf[3].cpu(), c["residual"][3])
    c["x"][torch.isnan(c["x"])] = 0
    c["w1"][E - 1] = 0
    check(c, buf[:T])
    c["residual"] = None
    assert (run(c)[0] == 0).all()


def test_an_expert_named_twice_counts_twice():
    c = case(31, 6, 4, 3, 64, 32, 48, F32)
    c["ids"][1] = torch.tensor([2, 2, 0])
    c["ids"][4] = torch.tensor([3, 3, 3])
    check(c, run(c))


def test_all_tokens_on_one_expert():
    for T in (16, 17, 64):
        c = case(41 + T, T, 8, 2, 128, 64, 64, BF16)
        c["ids"][:, 0], c["ids"][:, 1] = 5, -1
        check(c, run(c))


def test_nan_and_inf_stay_with_their_token():
    c = case(51, 20, 4, 2, 64, 32, 48, BF16)
    ref = run(c)
    c["x"][7, 3], c["x"][18, 9] = float("nan"), float("inf")
    y = run(c)
    keep = [t for t in range(20) if t not in (7, 18)]
    assert_bits_equal(y[keep], ref[keep], "other tokens")
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[18]).all()


def test_no_tokens_writes_nothing():
    c = case(61, 3, 4, 2, 64, 32, 48, BF16)
    c["x"], c["ids"], c["weights"] = c["x"][:0], c["ids"][:0], c["weights"][:0]
    y = torch.full((2, 48), 5.0, dtype=BF16, device=DEV)
    run(c, y=y)
    assert (y == 5).all()


def test_offsets_past_32_bits():
    """The last expert's weights lie past 2^32 elements' bytes from the first's."""
    E, K, F, N = 70, 8192, 4096, 16
    w1 = torch.empty(E, 2 * F, K, dtype=BF16, device=DEV)  # 9.4 GB
    w1[E - 1] = (torch.randn(2 * F, K, device=DEV) * K ** -0.5).to(BF16)
    w1[0] = 0
    c = case(71, 2, 1, 1, K, 8, N, BF16)
    c["ids"] = torch.tensor([[E - 1], [0]], dtype=torch.int32)
    c["weights"] = torch.ones(2, 1)
    w2 = (torch.randn(E, N, F, device=DEV) * F ** -0.5).to(BF16)
    y = run({"x": c["x"], "ids": c["ids"], "weights": c["weights"]}, w1=w1, w2=w2)
    x = c["x"][0].to(DEV).double()
    h = w1[E - 1].double() @ x
    ref = w2[E - 1].double() @ (torch.nn.functional.silu(h[:F]) * h[F:])
    assert (y[1] == 0).all()
    assert (y[0].double() - ref).abs().max() < 0.01 * ref.abs().max()


def test_deterministic_other_stream_and_graph_replay():
    c = case(81, 33, 12, 4, 128, 96, 72, BF16, bias=True, residual=True)
    ref = run(c)
    assert_bits_equal(run(c), ref, "again")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.full_like(ref, float("nan"))
    torch.cuda.synchronize()
    run(c, y=y, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert_bits_equal(y, ref, "other stream")
    d = {n: t.to(DEV) for n, t in c.items() if t is not None}
    ws = torch.empty(gl.gl_moe_few_tokens_workspace_size(33, 4, 12, 96), dtype=torch.uint8, device=DEV)
    kw = {n: d[n] for n in ("b1", "b2", "residual")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gl.gl_moe_few_tokens(d["x"], d["ids"], d["weights"], d["w1"], d["w2"], y, ws, **kw)
    for i in range(3):
        y.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert_bits_equal(y, ref, f"replay {i}")


def test_broken_weights_stay_with_their_tokens():
    """NaN and infinite weights of an expert reach the tokens that name it and no others."""
    for T in (5, 30, 50):
        c = case(91, T, 6, 2, 64, 40, 56, BF16)
        c["ids"][:, 0], c["ids"][:, 1] = 1, 2
        c["ids"][3, 1] = 4
        ref = run(c)
        c["w1"][4, 3, 5] = float("nan")
        c["w2"][4] = float("inf")
        y = run(c)
        keep = [t for t in range(T) if t != 3]
        assert_bits_equal(y[keep], ref[keep], "other tokens")
        assert not torch.isfinite(y[3]).any()
