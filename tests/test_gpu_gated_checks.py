"""The device-check build's gated layer and 8-bit integer products, in a child process (one library per
process), on the cases of gated_check_cases.py:

- valid launches: the checks stay silent (status 0) and every output is bit-identical to the
  product build's;
- a workspace whose last group has fewer rows than none: dW's tiles of that group are flagged and
  nothing is stored for them, neither in the group's own matrix nor in another's.  (A
  workgroup that starts after the flag writes nothing, so other tiles are right or untouched.)
"""
import os
import subprocess
import sys

import pytest
import torch

import gated_check_cases as cases
import grouped_gemm_gl_amd as gl
from gl_testutil import assert_bits_equal
from grouped_gemm_gl_amd import build as gl_build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STATUS_DEVICE_CHECK = 8  # GL_STATUS_DEVICE_CHECK


@pytest.fixture(scope="module")
def checked(tmp_path_factory):
    lib = gl_build.CHECKED_OUT
    assert os.path.exists(lib), f"{lib} is missing: build() makes it beside the library"
    out = str(tmp_path_factory.mktemp("gated_checks") / "results.pt")
    r = subprocess.run([sys.executable, "-u", os.path.join(ROOT, "tests", "gated_check_cases.py"), out], cwd=ROOT,
                       env=dict(os.environ, GL_LIBRARY_PATH=lib), stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True, timeout=100)
    print(r.stdout[-2000:], file=sys.stderr, flush=True)
    assert r.returncode == 0, r.stdout[-4000:]
    res = torch.load(out, weights_only=True)
    assert bytes(res.pop("library").tolist()).decode() == lib
    return res


def test_checked_build_is_silent_and_bit_identical(checked):
    gl.load()
    assert os.path.abspath(gl.library_path) != os.path.abspath(gl_build.CHECKED_OUT)
    mine = cases.run(gl)
    assert set(mine) == {k for k in checked if not k.startswith("tamper")}
    for k, v in mine.items():
        if k.endswith("_status"):
            assert int(v) == 0 and int(checked[k]) == 0, k
        else:
            assert_bits_equal(checked[k], v, f"{k}: device-check build vs product build")


@pytest.mark.parametrize("tile", sorted(cases.TAMPERED))
def test_checked_dw_flags_a_group_and_stores_nothing_for_it(checked, tile):
    ok, dw = checked[f"tamper_{tile}_ok"], checked[f"tamper_{tile}_dw"]
    assert int(checked[f"tamper_{tile}_status_ok"]) == 0 and bool(torch.isfinite(ok.float()).all())
    assert int(checked[f"tamper_{tile}_status"]) == STATUS_DEVICE_CHECK
    assert torch.isnan(dw[15].float()).all(), "the flagged group's matrix stays untouched"
    untouched = torch.isnan(dw[:15].float())
    assert bool((untouched | (dw[:15].view(torch.int16) == ok[:15].view(torch.int16))).all())
    # a tile is stored whole or not at all
    n, (rows, cols) = int(tile), dw.shape[1:]
    tiles = untouched.view(15, rows // n, n, cols // n, n).permute(0, 1, 3, 2, 4).flatten(3)
    assert bool((tiles.all(-1) == tiles.any(-1)).all())
