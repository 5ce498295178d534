"""Sets past what one launch can index are refused on the host: more than
2^31 - 1 tiles, of one tensor or of several together. The addresses stand for
nothing and are never read."""
import ctypes

import pytest

F32_TILE = 4096  # elements of a norm's tile


@pytest.fixture(scope="module")
def L():
    from ring_all_reduce_ddp_gb300 import build
    build.build_library()
    import ring_all_reduce_ddp_gb300 as d
    return d


def _create(L, numel, dtype=0):
    es = 4 if dtype == 0 else 2
    ptrs, at = [], 1 << 12
    for n in numel:
        ptrs.append(at)
        at += n * es
    h = ctypes.c_void_p(1)
    rc = L.lib().ddp_optim_create(ctypes.byref(h), len(numel), (ctypes.c_void_p * len(numel))(*ptrs),
                                  (ctypes.c_int64 * len(numel))(*numel), dtype)
    return rc, h, ptrs


@pytest.mark.parametrize("numel", [[1 << 46], [F32_TILE << 31], [F32_TILE << 30] * 2, [5, (F32_TILE << 31) - F32_TILE],
                                   [1 << 40] * 8])
def test_more_tiles_than_one_launch_has_blocks(L, numel):
    rc, h, _ = _create(L, numel)
    assert rc == L.DDP_ERR_ARG and h.value is None and "too large for one launch" in L.ddp_last_error()


@pytest.mark.gpu
def test_outputs_and_parameters_of_more_tiles_than_their_launch_has(L):
    """2^42 elements are 2^30 tiles of the norm, but 2^31 of the clip and 2^32
    of the update: the set calls refuse, and nothing is launched."""
    lib = L.lib()
    rc, h, ptrs = _create(L, [1 << 42])
    assert rc == L.DDP_OK
    launches = L.ddp_kernel_launches()
    far = [(ctypes.c_void_p * 1)((1 << 46) + (i << 45)) for i in range(3)]
    f = ctypes.c_void_p(0x800)  # apart from every range above
    for p, outs in ((1, far[0]), (3, (ctypes.c_void_p * 3)(*[x[0] for x in far]))):
        assert lib.ddp_optim_set_outputs(h, p, outs) == L.DDP_ERR_ARG
        assert "too large for one launch" in L.ddp_last_error()
    assert lib.ddp_optim_set_params(h, 1, far[0], 0, None, far[1], far[2], f) == L.DDP_ERR_ARG
    assert "overlap" not in L.ddp_last_error() and "too large for one launch" in L.ddp_last_error()
    assert lib.ddp_optim_clip(h, 0, 1.0, f, None) == L.DDP_ERR_STATE
    assert lib.ddp_optim_adamw(h, 1e-3, 0.9, 0.99, 1e-8, 0.0, None, 0.0, None) == L.DDP_ERR_STATE
    assert L.ddp_kernel_launches() == launches and lib.ddp_optim_destroy(h) == L.DDP_OK
