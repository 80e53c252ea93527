"""The rules that choose the gated layer's and the 8-bit integer products' kernels, on the host: the
cases of test_gpu_glu_choice.py take the kernels they name, and every kernel that some size takes has one.
A rule that moves a case to another kernel fails here."""
import math
import random
import shutil

import pytest
import torch

import glu_choice
import test_gpu_fp32_sums as sums
import test_gpu_gelu_tail as gelu
import test_gpu_glu_choice as cases
import test_gpu_int8_scales as scales

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host compiler")
NAME = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return glu_choice.build(str(tmp_path_factory.mktemp("choice")))


@pytest.mark.parametrize("what", ["glu", "dx", "dw"])
def test_cases_take_the_kernels_they_name(exe, what):
    table = {"glu": cases.FORWARD, "dx": cases.DX, "dw": cases.DW}[what]
    labels = [c[0] for c in table]
    q = [(what, NAME[t], len(m), sum(m), K, F, False) for _, t, m, K, F in table]
    assert glu_choice.ask(exe, q) == labels
    if what == "dw":  # gradients of fp32 too
        assert glu_choice.ask(exe, [("dw32", *r[1:]) for r in q]) == labels


def test_int8_cases_take_the_kernels_they_name(exe):
    for plain in (True, False):
        q = [("glu", "int8", len(m), sum(m), K, N if plain else N // 2, plain) for _, m, K, N in cases.INT8]
        assert glu_choice.ask(exe, q) == [c[0] for c in cases.INT8]


def test_other_tests_sizes_take_the_kernels_they_name(exe):
    """Of one group each: scales, fp32 sums, GELU's tail."""
    q = [("glu", "int8", 1, T, scales.K, N, True) for T, N in scales.SIZES.values()]
    assert glu_choice.ask(exe, q) == list(scales.SIZES)
    q = [("glu", "f32", 1, *s, False) for s in sums.FORWARD.values()]
    assert glu_choice.ask(exe, q) == list(sums.FORWARD)
    q = [("dx", "f32", 1, *s, False) for s in sums.DX.values()]
    assert glu_choice.ask(exe, q) == list(sums.DX)
    q = [("glu", "f16", 1, T, gelu.K, F, False) for T, F in gelu.SIZES]
    assert glu_choice.ask(exe, q) == ["32x32 parts", "32x32 parts", "256 full"]


def test_every_kernel_has_a_case(exe):
    rng = random.Random(0)

    def size(lo, hi, step):
        return max(step, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)

    sizes = [(size(1, 300, 1), size(1, 40000, 1), size(16, 20000, 16), size(8, 20000, 8)) for _ in range(40000)]
    for what, table in (("glu", cases.FORWARD), ("dx", cases.DX), ("dw", cases.DW), ("dw32", cases.DW)):
        for wide, types in ((False, ("bf16", "f16")), (True, ("f32",))):
            have = {c[0] for c in table if (c[1] == torch.float32) == wide}
            for t in types:
                took = set(glu_choice.ask(exe, [(what, t, *s, False) for s in sizes]))
                assert took <= have, (what, t, took - have)
    for plain in (False, True):
        took = set(glu_choice.ask(exe, [("glu", "int8", *s, plain) for s in sizes]))
        assert took <= {c[0] for c in cases.INT8}, took
