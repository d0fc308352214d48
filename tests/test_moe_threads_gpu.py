"""The mixture-of-experts products called from several host threads, each with its own stream,
workspace and sizes."""
import ctypes
import threading

import numpy as np
import pytest

from _native import compile_library
from test_moe_gpu import act, cuda, tq  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


class Job:
    """A product and its buffers; what it gives on the calling thread is in `want`."""

    def __init__(self, tq, experts, n, k, rows, seed):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed)
        codes = torch.randint(0, 256, (experts, n, k // 8), dtype=torch.uint8, device="cuda", generator=gen)
        scales = torch.ones((experts, n, k // 128), dtype=torch.float16, device="cuda")
        self.tq, self.w, self.stream = tq, tq.PackedExperts(codes, scales, experts, n, k, 1), torch.cuda.Stream()
        slots = experts * rows
        self.q, self.s = (cuda(a) for a in act(slots, k, seed=seed))
        order = cuda(np.arange(slots, dtype=np.int32))
        self.plan = tq.MoePlan(cuda(np.arange(experts + 1, dtype=np.int32) * rows), order, order)
        self.ws = torch.zeros(256 + slots * (2 * k + 16 * -(-k // 512)), dtype=torch.uint8, device="cuda")
        self.y = torch.empty((slots, n), device="cuda")
        self.want = tq.moe_gemv(self.w, self.q, self.s, self.plan, workspace=self.ws)
        torch.cuda.synchronize()

    def call(self):
        self.tq.moe_gemv(self.w, self.q, self.s, self.plan, y=self.y, workspace=self.ws, stream=self.stream)


def _run(targets):
    errors = []

    def guarded(target):
        try:
            target()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(t,)) for t in targets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


# (experts, n, k, rows per expert): the split, the stream and the tile kernel
SPLIT, STREAM, TILE = (2, 64, 256, 1), (64, 1000, 256, 1), (2, 64, 256, 100)


@pytest.mark.parametrize("size", [SPLIT, STREAM, TILE], ids=["split", "stream", "tile"])
def test_the_first_cuda_call_of_a_thread(tq, size):  # noqa: F811
    """A thread that has made no CUDA call before has no context yet."""
    import torch
    job = Job(tq, *size, seed=1)
    _run([job.call])
    torch.cuda.synchronize()
    assert torch.equal(job.y, job.want)


def test_the_first_cuda_call_of_a_thread_is_a_dense_product(tq):  # noqa: F811
    import torch
    from ternary_weight_dp4a_gb300 import synth
    codes, scales = synth.weight(256, 256, 0, 1, device="cuda")
    w = tq.pack_weights(codes, 0, scales)
    q, s = tq.rotate_quant(torch.randn((2, 256), device="cuda").bfloat16())
    ws, y, stream = tq.gemv_workspace(2, 256, 256), torch.empty((2, 256), device="cuda"), torch.cuda.Stream()
    want = tq.gemv(w, q, s, workspace=ws)
    torch.cuda.synchronize()
    _run([lambda: tq.gemv(w, q, s, y=y, workspace=ws, stream=stream)])
    torch.cuda.synchronize()
    assert torch.equal(y, want)


class _Product(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("slots", ctypes.c_int32), ("y", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


# the shared memory that a launch asks for differs with k and the rows: 64 and 1 KB on the
# split kernel, 125 and 60 on the stream kernel
@pytest.mark.parametrize("sizes", [((1, 64, 4096, 2), (1, 64, 128, 1)), ((64, 1000, 4096, 8), (64, 1000, 128, 1))],
                         ids=["split", "stream"])
def test_threads_with_different_sizes(tq, sizes, tmp_path):  # noqa: F811
    """No thread's launch depends on what another thread's call sets for the same kernel."""
    import torch
    lib = compile_library("threads", tmp_path)
    jobs = [Job(tq, *size, seed=i) for i, size in enumerate(sizes)]
    weights = [job.w.c_struct() for job in jobs]
    products = (_Product * len(jobs))(*[
        _Product(ctypes.addressof(w), job.q.data_ptr(), job.s.data_ptr(), job.plan.offsets.data_ptr(), job.plan.slots,
                 job.y.data_ptr(), job.ws.data_ptr(), job.ws.numel(), job.stream.cuda_stream)
        for w, job in zip(weights, jobs)])
    failed = lib.call_from_threads(ctypes.cast(tq.load().tq_moe_gemv, ctypes.c_void_p), products, len(jobs), 20000)
    torch.cuda.synchronize()
    assert failed == 0
    for job in jobs:
        assert torch.equal(job.y, job.want)
