"""The expert layer for a few tokens where its values leave the middle of their types'
ranges, against the float64 oracle.

The bound is the one derived in test_gpu_moe_few_tokens.py for the fp32 sums and the
output's rounding, with what is lost of a, the value between the products, by itself: 2^-16
of it (at least 16 significant bits) and, for fp16 products, 2^-48 of the token's largest;
nothing absolute, however small a is.
"""
import numpy as np
import pytest
import torch

import oracle
from gl_testutil import to64
from oracle import expert_block as eb
from test_gpu_moe_few_tokens import BF16, E24, F16, F32, U, case, dense, run

pytestmark = pytest.mark.gpu


def limits(c):
    """(reference, limit) of every output, limit without any absolute term but the output's."""
    x, ids, w, w1, w2 = to64(c["x"]), c["ids"].numpy(), to64(c["weights"]), dense(c, "w1"), dense(c, "w2")
    K, F, dtype = w1.shape[2], w2.shape[2], c["x"].dtype
    ref = eb.moe(x, ids, w, w1, w2)
    lim = np.zeros_like(ref)
    for t, j in np.ndindex(ids.shape):
        e = ids[t, j]
        if e < 0 or e >= len(w1) or w[t, j] == 0:
            continue
        h = w1[e] @ x[t]
        dh = (K + 8) * E24 * (np.abs(w1[e]) @ np.abs(x[t]))
        g, u = h[:F], h[F:]
        silu = np.abs(oracle.silu(g))
        a = silu * np.abs(u)
        da = 1.1 * (np.abs(u) + dh[F:]) * dh[:F] + silu * dh[F:] + (32 + np.abs(g)) * E24 * a
        da = da + (0 if dtype == F32 else 2.0 ** -16) * a + (2.0 ** -48 * a.max() if dtype == F16 else 0)
        lim[t] += w[t, j] * (np.abs(w2[e]) @ (da + (F + 80) * E24 * a))
    return ref, lim + U[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == F16 else 0)


def check(c):
    y = to64(run(c))
    ref, lim = limits(c)
    bad = ~(np.abs(y - ref) <= lim)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, worst {np.max(np.abs(y - ref) / (lim + 1e-300)):.3g} times"
    return ref


# one token and two (dot products), four, one MFMA step of tokens and several, both row counts of a workgroup
SHAPES = [(1, 3, 2, 72, 520, 40), (2, 3, 2, 64, 264, 4104), (4, 3, 2, 40, 72, 136), (3, 2, 1, 64, 1112, 24),
          (9, 2, 1, 72, 328, 4096), (20, 4, 3, 64, 136, 48), (64, 2, 2, 40, 264, 72)]


@pytest.mark.parametrize("T,E,k,K,F,N", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_large_values_between_the_products(T, E, k, K, F, N, dtype):
    """a of about 10^5, many past fp16's 65504, and outputs well inside every type."""
    c = case(T + N, T, E, k, K, F, N, dtype)
    c["w1"], c["w2"] = c["w1"] * 400, (c["w2"].float() * 1e-2).to(dtype)
    ref = check(c)
    assert 1 < np.abs(ref).max() < 60000


@pytest.mark.parametrize("T,E,k,K,F,N", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_small_values_between_the_products(T, E, k, K, F, N, dtype):
    """a of about 10^-7 under weights of about 10^3."""
    c = case(T + N + 1, T, E, k, K, F, N, dtype)
    c["x"], c["w2"] = (c["x"].float() * 2.0 ** -11).to(dtype), (c["w2"].float() * 2000 * F ** 0.5).to(dtype)
    ref = check(c)
    assert 1e-4 < np.abs(ref).max() < 1


@pytest.mark.parametrize("T,E,k,K,F,N", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_small_gates_and_tokens_of_many_sizes(T, E, k, K, F, N, dtype):
    """Weights of the slots from 10^-6 to 1 and tokens of 2^-9 to 2^5 beside one another."""
    c = case(T + N + 2, T, E, k, K, F, N, dtype)
    c["weights"] = 10.0 ** -(6 * torch.rand(c["weights"].shape, generator=torch.Generator().manual_seed(T)))
    c["x"] = (c["x"].float() * torch.exp2((torch.arange(T) * 5 % 15 - 9).float())[:, None]).to(dtype)
    c["w2"] = (c["w2"].float() * 30).to(dtype)
    check(c)


@pytest.mark.parametrize("T", [1, 2, 4, 20])
def test_one_column_far_above_the_others(T):
    """fp16: a row of a with one value 2^25 times the others keeps the others' bits: the large
    one meets weights of 0, so that only they are left in y."""
    K, F, N = 32, 264, 40
    c = case(7, T, 2, 1, K, F, N, F16)
    c["x"] = torch.full((T, K), 2.0 ** -5, dtype=F16)
    c["w1"] = (c["w1"].float() * 0.05).to(F16)
    c["w1"][:, 100], c["w1"][:, F + 100] = 200.0, 200.0
    c["w2"] = (c["w2"].float() * 3000).to(F16)
    c["w2"][:, :, 100] = 0
    ref = check(c)
    assert 2.0 ** -12 < np.abs(ref).max() < 60000


@pytest.mark.parametrize("T,E,k,K,F,N", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_infinite_weights_give_what_the_formula_gives(T, E, k, K, F, N, dtype):
    """Single infinite weights of W2, of both signs and in one row also two of them: infinities
    of the right sign, NaN where they meet with opposite signs, and all else as without them."""
    c = case(T + N + 3, T, E, k, K, F, N, dtype)
    clean, lim = limits(c)
    for n, f, v in ((0, 3, np.inf), (1, F - 1, -np.inf), (5, 9, np.inf), (5, F // 2, np.inf), (N - 1, F - 8, -np.inf)):
        c["w2"][1, n, f] = v
    y = to64(run(c))
    with np.errstate(invalid="ignore"):
        ref = eb.moe(to64(c["x"]), c["ids"].numpy(), to64(c["weights"]), to64(c["w1"]), to64(c["w2"]))
    finite = np.isfinite(ref)
    assert (~finite).any() or not (c["ids"] == 1).any()
    assert np.array_equal(y[~finite], ref[~finite], equal_nan=True)
    assert (np.abs(y - clean) <= lim)[finite].all()


@pytest.mark.parametrize("T", [1, 2, 4, 20])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_infinite_values_between_the_products(T, dtype):
    """An infinite weight of W1's second half: a is infinite in one column."""
    c = case(3, T, 2, 1, 64, 72, 40, dtype)
    c["w1"][1, 72 + 7, 5] = np.inf
    y = to64(run(c))
    with np.errstate(invalid="ignore"):
        ref = eb.moe(to64(c["x"]), c["ids"].numpy(), to64(c["weights"]), to64(c["w1"]), to64(c["w2"]))
    hit = c["ids"][:, 0].numpy() == 1
    assert np.isinf(ref[hit]).all() and np.array_equal(y[hit], ref[hit]) and np.isfinite(y[~hit]).all()


def test_misaligned_matrices_of_an_expert_are_refused():
    """Per-expert weights off a 16-byte boundary, scales off a 4-byte one: refused on the host."""
    for mx, name, off in ((False, "w1", 1), (False, "w2", 4), (True, "w1", 8), (True, "w1_scale", 2), (True, "w2_scale", 1)):
        c = case(1, 3, 2, 1, 64, 64, 32, BF16, mx=mx)
        names = ["w1", "w2"] + (["w1_scale", "w2_scale"] if mx else [])
        lists = {n: [t.cuda().clone() for t in c[n]] for n in names}
        run(c, **lists)
        t = lists[name][1]
        lists[name][1] = torch.cat([t.reshape(-1), t.reshape(-1)])[off:off + t.numel()].view(t.shape)
        with pytest.raises(ValueError, match=f"{name} must be"):
            run(c, **lists)


@pytest.mark.parametrize("T,N", [(1, 2048), (1, 2056), (1, 4088), (1, 4096), (2, 2048), (2, 2056), (9, 2040), (9, 2056), (20, 2064)])
@pytest.mark.parametrize("dtype,mx", [(F16, False), (BF16, False), (F32, False), (BF16, True)])
def test_output_widths_where_the_workgroups_change(T, N, dtype, mx):
    c = case(T + N + 4, T, 3, 2, 64, 96, N, dtype, mx=mx)
    check(c)
