"""A handle's tables are in device memory when the call that makes them
returns (GPU): a launch on a non-blocking stream, which nothing orders behind
the legacy stream that carries the upload, reads them whole. The legacy stream
is kept busy for a few tens of milliseconds meanwhile; a call that returned
before its upload had run would return before that work has."""
import math

import pytest

from oracle import optim as oo
from test_gpu_optim import HYPER, SIZES, U, Arena, Model

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Busy:
    """Work on the legacy default stream, and whether all of it is done."""

    def __init__(self):
        assert torch.cuda.current_stream().cuda_stream == 0
        self.x = torch.zeros(1 << 26, device="cuda")
        torch.cuda.synchronize()
        for _ in range(400):  # half a gigabyte of traffic each
            self.x += 1.0
        self.end = torch.cuda.Event()
        self.end.record()

    def done(self):
        return self.end.query()


def test_first_set_outputs_is_ordered_before_a_clip_on_another_stream():
    M = Model(50, SIZES, "bf16", "bf16", True, p=2)
    outs = [Arena([x * 0 + 1 for x in M.g.host], "bf16") for _ in range(2)]
    side, norm = torch.cuda.Stream(), torch.zeros((), device="cuda")
    busy = Busy()
    M.opt.set_outputs([o.views for o in outs])
    assert busy.done()
    M.opt.clip(math.inf, norm, stream=side)
    side.synchronize()
    for o in outs:  # nothing clipped: the gradients' bits
        assert all((a == b).all() for a, b in zip(o.now(), M.g.host)) and o.guards_intact()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_first_set_params_is_ordered_before_an_update_on_another_stream(kind):
    import ring_all_reduce_ddp_gb300 as D
    M = Model(51, SIZES, "f32", kind, kind == "bf16", p=8)
    before = M.snapshot()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    M.opt = D.DDPOptim(M.g.views)  # a handle without parameters yet
    busy = Busy()
    M.opt.set_params([x.views for x in M.params], M.m.views, M.v.views, M.step,
                     master=M.master.views if M.master else None)
    assert busy.done()
    M.opt.adamw(stream=side, **HYPER)
    side.synchronize()
    assert int(M.step) == 4
    M.check(before, 3)


def test_create_is_ordered_before_a_norm_on_another_stream():
    import ring_all_reduce_ddp_gb300 as D
    M = Model(52, SIZES)
    side, norm = torch.cuda.Stream(), torch.zeros((), device="cuda")
    busy = Busy()
    opt = D.DDPOptim(M.g.views)
    assert busy.done()
    opt.norm(norm, stream=side)
    side.synchronize()
    want = oo.norms(M.g.host)[0]
    assert abs(float(norm) - want) <= 33 * U * want


@pytest.mark.parametrize("buffers", [False, True])
def test_a_reducer_is_made_before_its_step_on_another_stream(buffers):
    """Integers: every sum is exact, whatever its order."""
    import ring_all_reduce_ddp_gb300 as D
    p, sizes = 4, [5000, 1, 0, 70001, 33]
    g = torch.Generator().manual_seed(53)
    grads = [[torch.randint(-99, 100, (n,), generator=g).float().cuda() for n in sizes] for _ in range(p)]
    bufs = [[torch.full((77,), float(r), device="cuda")] for r in range(p)]
    want = [sum(grads[r][j] for r in range(p)) for j in range(len(sizes))]
    side = torch.cuda.Stream()
    busy = Busy()
    red = D.DDPReducer(grads)
    assert busy.done()
    if buffers:
        red.set_buffers(bufs, root=1)
    red.step(1.0, stream=side)
    side.synchronize()
    for r in range(p):
        assert all(torch.equal(grads[r][j], want[j]) for j in range(len(sizes)))
        assert bool((bufs[r][0] == (1.0 if buffers else r)).all())
