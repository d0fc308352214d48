"""A bounded wait that runs out ends the kernel and sets the error word.  (Nothing faults: the copies
land, only their count is never complete.)"""
import ctypes
import time

import numpy as np
import pytest

from _native import compile_library
from test_moe_gpu import act, cuda, tq  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stalled(tmp_path_factory):
    lib = compile_library("stalled_copies", tmp_path_factory.mktemp("native"), "tq_tmap.cu")
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    lib.stalled_product.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp]
    return lib


@pytest.mark.parametrize("fmt", [0, 1])
def test_the_stream_kernel_ends_when_its_copies_do_not(tq, stalled, fmt):  # noqa: F811
    """Each warp waits half a second for its first stage, and as long for the one or two behind it, and
    for no more: a warp that went on waiting would wait for all stages of its units, 8 for each."""
    import torch
    experts, n, k, rows = 64, 1000, 4096, 2
    codes = torch.zeros((experts, n, k // (4 if fmt == 0 else 8)), dtype=torch.uint8, device="cuda")
    scales = torch.ones((experts, n, k // 128), dtype=torch.float16, device="cuda")
    q, s = (cuda(a) for a in act(experts * rows, k))
    offsets = cuda(np.arange(experts + 1, dtype=np.int32) * rows)
    y = torch.full((experts * rows, n), -1.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bits = ctypes.c_uint32(0)
    assert stalled.lost_waits(ctypes.byref(bits)) == 0 and bits.value in (0, 1 << 12)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert stalled.stalled_product(codes.data_ptr(), scales.data_ptr(), experts, n, k, fmt, q.data_ptr(), s.data_ptr(),
                                   offsets.data_ptr(), experts * rows, y.data_ptr(), err.data_ptr()) == 0
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert int(err) == 1 << 12 and (y == -1.0).all()
    assert 0.2 < took < 5.0, took
    del err                                                          # the bit outlives the caller's word
    assert stalled.lost_waits(ctypes.byref(bits)) == 0 and bits.value == 1 << 12
    # the device is as usable as before
    w = tq.PackedExperts(codes, scales, experts, n, k, fmt)
    order = cuda(np.arange(experts * rows, dtype=np.int32))
    got = tq.moe_gemv(w, q, s, tq.MoePlan(offsets, order, order))
    assert torch.isfinite(got).all() and (got != -1.0).all()
    assert tq.moe_read_error_word() == 0                             # (the word of the library, not of this test's copy)
