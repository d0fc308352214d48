"""A bounded wait of the 4-bit tile kernel that runs out ends the call, whatever its size, and sets the error word.
(Nothing faults: the copies land, only their count is never complete.)"""
import ctypes
import time

import pytest

from _native import compile_library
from test_q4_gpu import Matrix, _x, tq  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

KNOWN = 0x3ff                                                        # the bits that include/tq_q4.h names


@pytest.fixture(scope="module")
def native(tmp_path_factory):
    lib = compile_library("stalled_tile", tmp_path_factory.mktemp("native"), "tq_tmap.cu")
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    lib.set_stall.argtypes = [ctypes.c_uint32]
    lib.product.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp]
    return lib


class Call:
    """One product by the library of this test; y stays the same tensor."""

    def __init__(self, tq, native, n, k, group, mins, m):  # noqa: F811
        import torch
        self.w, self.x, self.native = Matrix(tq, n, k, group, mins, 1), _x(m, k, 2), native
        self.want = tq.q4_gemv(self.w.dev, self.x)
        self.y = torch.empty((m, n), device="cuda")
        self.ws = torch.empty(tq.q4_workspace_bytes(m, k, group), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

    def __call__(self):
        import torch
        d = self.w.dev
        assert self.native.product(d.codes.data_ptr(), d.scales.data_ptr(), 0 if d.mins is None else d.mins.data_ptr(), d.n, d.k,
                                   d.group, self.x.data_ptr(), len(self.x), self.y.data_ptr(), self.ws.data_ptr(),
                                   torch.cuda.current_stream().cuda_stream) == 0

    def stalled(self, run):
        """The seconds that run takes over copies that never complete."""
        import torch
        assert self.native.set_stall(16) == 0
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        run()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        assert self.native.set_stall(0) == 0
        bits = ctypes.c_uint32(0)
        assert self.native.lost_waits(ctypes.byref(bits)) == 0
        assert bits.value & 1 << 6 and bits.value & ~(1 << 6) and not bits.value & ~KNOWN, hex(bits.value)
        return took

    def right(self, run):
        import torch
        self.y.fill_(-1.0)
        run()
        torch.cuda.synchronize()
        return torch.equal(self.y, self.want)


# Rounds of tiles (152 run at once): one, split along k over eight CTAs; one; seven; six, and a launch of its own for the rest
SIZES = [(1000, 2048), (9000, 512), (130_000, 512), (120_000, 1024)]


@pytest.mark.parametrize("group,mins,m", [(128, False, 40), (128, True, 100), (32, False, 100), (32, True, 100), (64, True, 20)])
@pytest.mark.parametrize("n,k", SIZES)
def test_a_call_ends_when_its_copies_do_not(tq, native, n, k, group, mins, m):  # noqa: F811
    """Half a second for the first wait and as long for the copies in flight, in the first round of tiles of each launch;
    later rounds do not wait again (seven rounds of this, with two seconds for four stages in flight, took 17 s)."""
    call = Call(tq, native, n, k, group, mins, m)
    took = call.stalled(call)
    print(f"{took:.2f} s")
    assert 0.2 < took < (3.5 if k == 1024 else 1.8), took
    assert call.right(call)                                          # the device is as usable as before, all rounds
    took = call.stalled(call)                                        # and another call waits for itself
    assert 0.2 < took < (3.5 if k == 1024 else 1.8), took
    assert call.right(call)
    assert tq.q4_read_error_word() == 0                              # (the word of the library, not of this test's copy)


@pytest.mark.parametrize("n,k", SIZES)
def test_a_replay_after_one_that_was_lost_is_right(tq, native, n, k):  # noqa: F811
    import torch
    call = Call(tq, native, n, k, 128, False, 40)
    assert native.set_stall(0) == 0 and call.right(call)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        assert 0.2 < call.stalled(g.replay) < (3.5 if k == 1024 else 1.8)
        for _ in range(3):
            assert call.right(g.replay)
