"""The clip coefficient's edges in oracle/optim.py (CPU)."""
import math

import numpy as np

from oracle import optim as oo


def test_an_infinite_limit_clips_nothing():
    for norm in (0.0, 1.0, 1e300, math.inf):
        assert oo.coefficient(norm, math.inf) == 1.0
    assert math.isnan(oo.coefficient(math.nan, math.inf))
    x = [np.array([np.inf, -2.0]), np.array([0.5])]
    for kind in ("l2", "inf"):
        n, y = oo.clip(x, math.inf, kind)
        assert n == math.inf and all(np.array_equal(a, b) for a, b in zip(x, y))
