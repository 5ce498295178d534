"""Which stream a DDPOptim call takes when none is given (GPU): the current
one, with and without the raw accessor that saves building a stream object."""
import pytest

import ring_all_reduce_ddp_gb300 as D

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [True, False])
def test_calls_default_to_the_current_stream(raw, monkeypatch):
    if not raw:  # a torch without the accessor
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    g = torch.full((10000,), 0.5, device="cuda")
    opt = D.DDPOptim([g])
    norm = torch.zeros((), device="cuda")
    assert opt._on(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert opt._on(None) == side.cuda_stream
        opt.norm(norm)
    side.synchronize()
    assert float(norm) == 50.0
