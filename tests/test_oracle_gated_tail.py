"""The oracle's GELU in its negative tail, where 1 + erf would cancel."""
import math

import numpy as np
import pytest

from oracle import gated


def test_gelu_keeps_its_negative_tail():
    # Phi(-3), Phi(-6), Phi(-9) to the digits that tables of the normal distribution give
    for v, phi in ((-3.0, 1.349898031630095e-3), (-6.0, 9.865876450376981e-10), (-9.0, 1.1285884059538405e-19)):
        assert gated.act("gelu", v) == pytest.approx(v * phi, rel=1e-12, abs=0)
        density = math.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
        assert gated.slope("gelu", v) == pytest.approx(phi + v * density, rel=1e-12, abs=0)


def test_gelu_keeps_its_middle_and_its_limits():
    v = np.array([0.0, 0.5, 3.0, 40.0])
    for a, b in zip(gated.act("gelu", v), v):
        assert a == pytest.approx(b * 0.5 * math.erfc(-b / math.sqrt(2.0)), rel=1e-14, abs=0)
    assert gated.act("gelu", -40.0) == 0 and gated.slope("gelu", -40.0) == 0 and gated.slope("gelu", 40.0) == 1
