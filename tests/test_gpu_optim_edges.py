"""The clip's coefficient where norm and limit are infinite (GPU): a limit of
infinity means that nothing is clipped, whatever the norm, unless it is NaN."""
import math

import numpy as np
import pytest

import ring_all_reduce_ddp_gb300 as D
from oracle import optim as oo
from test_gpu_optim import SIZES, Arena, _values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KIND = {"l2": D.DDP_NORM_L2, "inf": D.DDP_NORM_INF}


def _clipped(x, dtype, kind, limit):
    g = Arena(x, dtype, 1)
    outs = [Arena([np.ones(a.size) for a in x], dtype, o) for o in (1, 2)]  # one misaligned: element by element
    norm, got = torch.zeros((), device="cuda"), []
    for o in outs:
        opt = D.DDPOptim(g.views)
        opt.set_outputs([o.views])
        opt.clip(limit, norm, KIND[kind])
        got.append(o.now())
        assert o.guards_intact()
    return g, float(norm), got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_an_infinite_limit_keeps_infinite_gradients(kind, dtype):
    x = _values(np.random.default_rng(61), SIZES)
    x[-1][17], x[-2][0] = np.inf, -np.inf
    g, norm, got = _clipped(x, dtype, kind, math.inf)
    assert norm == math.inf and oo.coefficient(norm, math.inf) == 1.0
    for out in got:
        assert all(np.array_equal(a, b) for a, b in zip(out, g.host))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_infinite_limit_keeps_gradients_whose_norm_is_past_fp32(dtype):
    """Finite gradients of 3e38: the norm of 5,000 of them rounds to infinity."""
    x = [np.full(5000, 3e38, np.float32), np.full(7, -1.0, np.float32)]
    g, norm, got = _clipped(x, dtype, "l2", math.inf)
    assert norm == math.inf
    for out in got:
        assert all(np.array_equal(a, b) for a, b in zip(out, g.host))


@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_a_nan_stays_one_under_an_infinite_limit(kind):
    x = _values(np.random.default_rng(62), [50, 5000])
    x[1][17] = np.nan
    _, norm, got = _clipped(x, "f32", kind, math.inf)
    assert math.isnan(norm) and math.isnan(oo.coefficient(norm, math.inf))
    for out in got:
        assert all(np.isnan(a).all() for a in out)
