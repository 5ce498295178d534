"""The norm, clip and update of sets past the small ones' size (GPU), against
oracle/optim.py in fp64: updates of more than 1,024 tiles, whose scalars come
from a launch of their own, and norms whose blocks walk several full tiles.

Bounds, derived from the arithmetic (u = 2^-24, one fp32 rounding):
  norm   fp32 sums of at most 32 squares (32 u, halved by the root), fp64
         beyond, the sum's rounding (halved) and the root's: 17.5 u, and half a
         unit for fp64's sums: 18 u relative.
  c      the norm's, an addition and a division: 20 u.
  clip   c's and the product's rounding: 21 u relative, and the smallest fp32
         subnormal where products underflow.
  adamw  as Model.check derives it, from g' = c g that is 21 u off.
Stored bf16 values are the rounding of a value within the fp32 bound."""
import math

import numpy as np
import pytest

import ring_all_reduce_ddp_gb300 as D
from oracle import optim as oo
from test_gpu_optim import HYPER, SIZES, U, Arena, Model, _stored_ok, _values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TILE = 1024                                # elements of an update's tile
BEGUN = 1024                               # tiles of the largest update in one launch
LARGE = SIZES + [700_001, 0, 600_007, 5]   # 1,412 tiles, full and ragged ones
OFF_C = 21 * U
TYPES = [("f32", "f32", False), ("bf16", "bf16", True), ("bf16", "bf16", False), ("f32", "bf16", True),
         ("f32", "bf16", False), ("bf16", "f32", False)]
KIND = {"l2": D.DDP_NORM_L2, "inf": D.DDP_NORM_INF}


def _norms(host, kind="l2"):
    """(norm, [norm of each]) in fp64, by numpy's sums."""
    if kind == "inf":
        each = [float(np.abs(x.astype(np.float64)).max()) if x.size else 0.0 for x in host]
        return max(each), each
    sums = [float(np.square(x.astype(np.float64)).sum()) for x in host]
    return math.sqrt(math.fsum(sums)), [math.sqrt(s) for s in sums]


def _norm_ok(got, want):
    return abs(got - want) <= 18 * U * want + 2.0 ** -149


def _scalar():
    return torch.full((), -1.0, dtype=torch.float32, device="cuda")


def _launches(f, *a, **k):
    n = D.ddp_kernel_launches()
    f(*a, **k)
    return D.ddp_kernel_launches() - n


def _small_tensors(seed):
    """3,001 tensors of up to 2,999 elements, some 6,000 tiles."""
    return [int(x) for x in np.random.default_rng(seed).integers(0, 3000, size=3001)]


# ------------------------------------------------------------ the update
@pytest.mark.parametrize("offs", [(0, 0, 0), (1, 0, 0), (3, 3, 3), (0, 0, 5)])
@pytest.mark.parametrize("p", [1, 3])
@pytest.mark.parametrize("gdt,pdt,master", TYPES)
def test_large_update(gdt, pdt, master, p, offs):
    """Aligned; the gradients alone misaligned; all alike off a boundary; the
    parameters alone, where all streams go element by element."""
    M = Model(71, LARGE, gdt, pdt, master, p, offs)
    for t in (3, 4):
        before = M.snapshot()
        assert _launches(M.opt.adamw, **HYPER) == 2
        assert int(M.step) == t + 1
        M.check(before, t)
    assert all(np.array_equal(a, b) for a, b in zip(M.g.now(), M.g.host))


@pytest.mark.parametrize("gdt,pdt,master", TYPES)
@pytest.mark.parametrize("share", [0.2, 3.0])
def test_large_update_clipped_by_the_norm(share, gdt, pdt, master):
    M = Model(72, LARGE, gdt, pdt, master, p=2, offs=(7, 0, 0))
    norm = _scalar()
    n = _norms(M.g.host)[0]
    limit = float(np.float32(share * n))
    before = M.snapshot()
    M.opt.norm(norm)
    M.opt.adamw(norm=norm, max_norm=limit, **HYPER)
    assert _norm_ok(float(norm), n) and int(M.step) == 4
    M.check(before, 3, c=oo.coefficient(n, limit), off_c=OFF_C)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("gdt,pdt,master", [("f32", "f32", False), ("bf16", "bf16", True)])
def test_large_update_skips_a_norm_that_is_not_finite_and_goes_on(gdt, pdt, master, bad):
    M = Model(73, LARGE, gdt, pdt, master, p=2)
    at = LARGE.index(600_007)
    M.g.views[at][600_006] = bad
    norm = _scalar()
    before = M.snapshot()
    for _ in range(3):
        M.opt.norm(norm)
        M.opt.adamw(norm=norm, max_norm=1.0, **HYPER)
    assert not math.isfinite(float(norm)) and int(M.step) == 3
    for a, b in zip(M.arenas()[1:], before[1:]):
        assert all(np.array_equal(x, y) for x, y in zip(a.now(), b)) and a.guards_intact()
    M.g.views[at][600_006] = 0.001
    before = M.snapshot()
    n = _norms(before[0])[0]
    M.opt.norm(norm)
    M.opt.adamw(norm=norm, max_norm=math.inf, **HYPER)
    assert int(M.step) == 4 and _norm_ok(float(norm), n)
    M.check(before, 3)


@pytest.mark.parametrize("tiles", [BEGUN, BEGUN + 1])
@pytest.mark.parametrize("gdt,pdt,master", [("f32", "f32", False), ("bf16", "bf16", True)])
def test_either_side_of_the_one_launch_limit(gdt, pdt, master, tiles):
    for sizes in ([(tiles - 1) * TILE + 1], [TILE] * 3 + [(tiles - 4) * TILE + 1, 0]):
        M = Model(74, sizes, gdt, pdt, master, p=2)
        norm = _scalar()
        n = _norms(M.g.host)[0]
        limit = float(np.float32(0.5 * n))
        M.opt.norm(norm)
        for t in (3, 4):
            before = M.snapshot()
            assert _launches(M.opt.adamw, norm=norm, max_norm=limit, **HYPER) == (1 if tiles <= BEGUN else 2)
            assert int(M.step) == t + 1
            M.check(before, t, c=oo.coefficient(n, limit), off_c=OFF_C)


@pytest.mark.parametrize("step", [0, 1, 10 ** 12])
@pytest.mark.parametrize("beta1,beta2", [(0.0, 0.0), (0.999, 0.9999)])
def test_large_update_bias_corrections(beta1, beta2, step):
    h = dict(HYPER, beta1=beta1, beta2=beta2)
    M = Model(75, LARGE, step=step)
    before = M.snapshot()
    M.opt.adamw(**h)
    assert int(M.step) == step + 1
    M.check(before, step, hyper=h)


def test_large_updates_in_a_row_agree_with_updates_that_wait():
    """The scalars' place is written again while the update before drains."""
    A, B = (Model(76, LARGE, "bf16", "bf16", True, p=2) for _ in range(2))
    na, nb = _scalar(), _scalar()
    rates = [1e-3 * (1 + i % 7) for i in range(40)]
    for lr in rates:
        A.opt.norm(na)
        A.opt.adamw(lr, norm=na, max_norm=1e-2)
    for lr in rates:
        B.opt.norm(nb)
        torch.cuda.synchronize()
        B.opt.adamw(lr, norm=nb, max_norm=1e-2)
        torch.cuda.synchronize()
    assert float(na) == float(nb) and int(A.step) == int(B.step) == 43
    for a, b in zip(A.arenas(), B.arenas()):
        assert torch.equal(a.base, b.base)


def test_large_update_captured_and_replayed():
    M = Model(77, LARGE, "f32", "bf16", True, p=2)
    norm = torch.zeros((), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.opt.norm(norm)
        M.opt.adamw(norm=norm, max_norm=0.125, **HYPER)
    at = LARGE.index(700_001)
    for t in (3, 4, 5):
        M.g.views[at].mul_(1.5)
        before = M.snapshot()
        n = _norms(before[0])[0]
        graph.replay()
        torch.cuda.synchronize()
        assert int(M.step) == t + 1 and _norm_ok(float(norm), n)
        M.check(before, t, c=oo.coefficient(n, 0.125), off_c=OFF_C)
    M.g.views[at][3] = math.nan  # a replay skips as a call does
    before = M.snapshot()
    graph.replay()
    torch.cuda.synchronize()
    assert int(M.step) == 6
    for a, b in zip(M.arenas()[1:], before[1:]):
        assert all(np.array_equal(x, y) for x, y in zip(a.now(), b))


@pytest.mark.parametrize("gdt,pdt,master", [("f32", "f32", False), ("bf16", "bf16", True)])
def test_update_of_thousands_of_tensors(gdt, pdt, master):
    M = Model(78, _small_tensors(7), gdt, pdt, master, p=2, offs=(1, 2, 2))
    norm = _scalar()
    n = _norms(M.g.host)[0]
    limit = float(np.float32(0.5 * n))
    before = M.snapshot()
    M.opt.norm(norm)
    assert _launches(M.opt.adamw, norm=norm, max_norm=limit, **HYPER) == 2
    M.check(before, 3, c=oo.coefficient(n, limit), off_c=OFF_C)


# ------------------------------------------------------- norm and clip
# 8.9 M elements: some 2,170 full fp32 tiles (1,085 in bf16) over 608 blocks.
WALK = [3, 5_000_011, 0, 4097, 3_000_001, 900_000, 17]


@pytest.mark.parametrize("off", [0, 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_norm_of_several_full_tiles_a_block(kind, dtype, off):
    g = Arena(_values(np.random.default_rng(81), WALK), dtype, off)
    opt = D.DDPOptim(g.views)
    norm, alone, each = _scalar(), _scalar(), torch.full((len(WALK),), -1.0, device="cuda")
    opt.norm(norm, each, KIND[kind])
    opt.norm(alone, kind=KIND[kind])
    want, parts = _norms(g.host, kind)
    assert float(norm) == float(alone)
    if kind == "inf":
        assert float(norm) == want and each.tolist() == parts
    else:
        assert _norm_ok(float(norm), want) and all(_norm_ok(a, b) for a, b in zip(each.tolist(), parts))
    for j, i in ((1, 0), (1, 5_000_010), (4, 1_234_567), (5, 899_999)):  # every element counts, and only once
        keep = g.views[j][i].clone()
        g.views[j][i] = 1000.0
        opt.norm(norm, each, KIND[kind])
        x = float(parts[j] ** 2 - float(keep) ** 2 + 1e6) if kind == "l2" else 1e6
        y = float(want ** 2 - float(keep) ** 2 + 1e6) if kind == "l2" else 1e6
        assert _norm_ok(float(each[j]), math.sqrt(x)) and _norm_ok(float(norm), math.sqrt(y))
        g.views[j][i] = math.nan
        opt.norm(norm, each, KIND[kind])
        assert math.isnan(float(norm)) and [math.isnan(v) for v in each.tolist()] == [q == j for q in range(len(WALK))]
        g.views[j][i] = keep


@pytest.mark.parametrize("goff,ooff", [(0, 0), (1, 0), (5, 5), (0, 1)])
@pytest.mark.parametrize("p", [1, 2, 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_large_clip(kind, dtype, p, goff, ooff):
    """Gradients off the outputs' boundaries among them, and either norm."""
    g = Arena(_values(np.random.default_rng(82), LARGE), dtype, goff)
    outs = [Arena([np.ones(n) for n in LARGE], dtype, ooff) for _ in range(p)]
    opt = D.DDPOptim(g.views)
    opt.set_outputs([o.views for o in outs])
    n = _norms(g.host, kind)[0]
    limit, norm = float(np.float32(0.3 * n)), _scalar()
    opt.clip(limit, norm, KIND[kind])
    c = oo.coefficient(n, limit)
    first = outs[0].now()
    for j, (a, x) in enumerate(zip(first, g.host)):
        y = c * x.astype(np.float64)
        assert _stored_ok(a, y, OFF_C * np.abs(y) + 2.0 ** -149, dtype).all(), j
    for o in outs:
        assert o.guards_intact() and all(np.array_equal(a, b) for a, b in zip(o.now(), first))
    assert all(np.array_equal(a, b) for a, b in zip(g.now(), g.host))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_large_clip_in_place(kind, dtype):
    """Replica 0's gradients are the handle's own, as after a sync."""
    g = Arena(_values(np.random.default_rng(83), LARGE), dtype, 2)
    other = Arena(_values(np.random.default_rng(83), LARGE), dtype, 2)
    opt = D.DDPOptim(g.views)
    opt.set_outputs([g.views, other.views])
    n = _norms(g.host, kind)[0]
    limit, norm = float(np.float32(0.1 * n)), _scalar()
    opt.clip(limit, norm, KIND[kind])
    c = oo.coefficient(n, limit)
    for j, (a, b, x) in enumerate(zip(g.now(), other.now(), g.host)):
        y = c * x.astype(np.float64)
        assert _stored_ok(a, y, OFF_C * np.abs(y) + 2.0 ** -149, dtype).all() and np.array_equal(a, b), j
    assert g.guards_intact() and other.guards_intact()
