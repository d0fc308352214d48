"""The entry points for 4-bit weights and sampling reject bad arguments before touching the GPU, and
the binding refuses tensors that the kernels could not read.  No GPU needed."""
import ctypes

import pytest

from ternary_weight_dp4a_gb300 import build as tqbuild
from ternary_weight_dp4a_gb300 import tq
from test_moe_binding import ELSEWHERE, HOST, Stream, Tensor, launched  # noqa: F401 (fixture)

OK, ARG, ALIGN = 0, 1, 2
ST = ctypes.c_void_p(0)


def P(a):
    return ctypes.c_void_p(a)


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    return tq.load()


def _w(codes=0x1000, scales=0x2000, mins=0, n=40, k=256, group=64):
    return tq._Q4(codes, scales, mins, n, k, group)


BAD = (dict(codes=0), dict(scales=0), dict(n=0), dict(n=(1 << 22) + 1), dict(k=0), dict(k=200), dict(k=32768 + 128),
       dict(group=16), dict(group=0), dict(group=256))


def test_sizes(lib):
    assert lib.tq_q4_codes_bytes(1, 128) == 16 * 64 and lib.tq_q4_codes_bytes(17, 256) == 32 * 128
    assert lib.tq_q4_scales_bytes(17, 256, 32) == 32 * 8 * 2 and lib.tq_q4_scales_bytes(16, 128, 128) == 32
    assert lib.tq_q4_codes_bytes(1 << 22, 32768) == 1 << 36                    # past 32 bits
    for n, k in ((0, 128), (-1, 128), (1, 0), (1, 64), (1, 32768 + 128), ((1 << 22) + 1, 128)):
        assert lib.tq_q4_codes_bytes(n, k) == 0 and lib.tq_q4_scales_bytes(n, k, 32) == 0
    for group in (0, 16, 96, 256, -32):
        assert lib.tq_q4_scales_bytes(16, 256, group) == 0


def test_pack_rejects(lib):
    def call(codes=0x1000, scales=0x2000, mins=0x3000, n=40, k=256, group=64, pc=0x4000, ps=0x5000, pm=0x6000):
        return lib.tq_q4_pack(P(codes), P(scales), P(mins), n, k, group, P(pc), P(ps), P(pm), ST)
    for bad in BAD + (dict(pc=0), dict(ps=0), dict(pm=0), dict(mins=0)):
        assert call(**bad) == ARG, bad
    for bad in (dict(codes=0x1004), dict(scales=0x2001), dict(mins=0x3001), dict(pc=0x4008), dict(ps=0x5008), dict(pm=0x6008)):
        assert call(**bad) == ALIGN, bad


def test_products_reject(lib):
    def gemv(w=_w(), x=0x7000, m=3, y=0x8000, t=0, ws=0, size=0):
        return lib.tq_q4_gemv(ctypes.byref(w) if w else None, P(x), m, P(y), t, P(ws), size, ST)

    def gateup(g=_w(), u=_w(), x=0x7000, m=3, h=0x8000, ws=0, size=0):
        return lib.tq_q4_gateup(ctypes.byref(g) if g else None, ctypes.byref(u) if u else None, P(x), m, P(h), P(ws), size, ST)
    assert gemv(w=None) == ARG and gateup(g=None) == ARG and gateup(u=None) == ARG
    for bad in BAD:
        assert gemv(w=_w(**bad)) == ARG and gateup(g=_w(**bad)) == ARG and gateup(u=_w(**bad)) == ARG, bad
    for bad in (dict(codes=0x1008), dict(scales=0x2008), dict(mins=0x3008)):
        assert gemv(w=_w(**bad)) == ALIGN and gateup(g=_w(**bad)) == ALIGN and gateup(u=_w(**bad)) == ALIGN, bad
    for call in (gemv, gateup):
        assert call(x=0) == ARG and call(m=0) == ARG and call(m=-1) == ARG and call(m=(1 << 20) + 1) == ARG
        assert call(x=0x7008) == ALIGN
    assert gemv(y=0) == ARG and gemv(t=2) == ARG and gemv(t=-1) == ARG and gemv(y=0x8002) == ALIGN and gemv(y=0x8001, t=1) == ALIGN
    assert gateup(h=0) == ARG and gateup(h=0x8001) == ALIGN
    m = 17                                                                  # minima: sums of x are needed
    mins, need = _w(mins=0x3000), lib.tq_q4_workspace_bytes(m, 256, 64)
    assert need == 32 * 4 * 4 and lib.tq_q4_workspace_bytes(16, 256, 64) == 0
    for bad in ((0, 256, 64), (17, 200, 64), (17, 256, 16), (1 << 21, 256, 64)):
        assert lib.tq_q4_workspace_bytes(*bad) == 0
    for call in (lambda **a: gemv(w=mins, m=m, **a), lambda **a: gateup(g=mins, u=mins, m=m, **a)):
        assert call() == ARG and call(ws=0x9010, size=need) == ALIGN and call(ws=0x9000, size=need - 1) == 4
    for other in (dict(n=41), dict(k=128), dict(group=32), dict(mins=0x3000)):
        assert gateup(u=_w(**other)) == ARG, other


def test_sample_rejects(lib):
    def call(l=0x1000, lt=0, m=2, v=10, t=0x2000, k=0x3000, p=0x4000, f=0x5000, u=0x6000, ids=0x7000, probs=0x8000):
        return lib.tq_sample(P(l), lt, m, v, P(t), P(k), P(p), P(f), P(u), P(ids), P(probs), ST)
    for bad in (dict(l=0), dict(u=0), dict(ids=0), dict(lt=2), dict(lt=-1), dict(m=0), dict(m=(1 << 20) + 1), dict(v=0),
                dict(v=(1 << 20) + 1)):
        assert call(**bad) == ARG, bad
    for bad in (dict(l=0x1002), dict(l=0x1001, lt=1), dict(t=0x2002), dict(k=0x3001), dict(p=0x4002), dict(f=0x5002),
                dict(u=0x6002), dict(ids=0x7002), dict(probs=0x8002)):
        assert call(**bad) == ALIGN, bad


def _tensors(torch):
    u8, i32, f32, f16, bf16 = torch.uint8, torch.int32, torch.float32, torch.float16, torch.bfloat16
    w = {"codes": (u8, 48 * 128), "scales": (f16, 48 * 4), "mins": (f16, 48 * 4)}
    up = {name + "2": kind for name, kind in w.items()}
    return {
        "pack": dict(codes=(u8, 40, 256), scales=(f16, 40, 4), mins=(f16, 40, 4)),
        "gemv": dict(w, x=(bf16, 3, 256), y=(f32, 3, 40), workspace=(u8, 4096)),
        "gateup": dict(w, **up, x=(bf16, 3, 256), h=(bf16, 3, 40), workspace=(u8, 4096)),
        "sample": dict(logits=(bf16, 3, 50), uniform=(f32, 3), temperature=(f32, 3), top_k=(i32, 3), top_p=(f32, 3),
                       min_p=(f32, 3), ids=(i32, 3), probs=(f32, 3)),
    }


def _call(op, t):
    w = lambda s="": tq.PackedQ4(t["codes" + s], t["scales" + s], t["mins" + s], 40, 256, 64)  # noqa: E731
    if op == "pack":
        return tq.pack_q4(t["codes"], t["scales"], t["mins"], stream=0)
    if op == "gemv":
        return tq.q4_gemv(w(), t["x"], y=t["y"], workspace=t["workspace"], stream=Stream())
    if op == "gateup":
        return tq.q4_gateup(w(), w("2"), t["x"], h=t["h"], workspace=t["workspace"], stream=Stream())
    return tq.sample(t["logits"], t["uniform"], t["temperature"], t["top_k"], t["top_p"], t["min_p"], ids=t["ids"],
                     probs=t["probs"], stream=Stream())


@pytest.mark.parametrize("op", ["pack", "gemv", "gateup", "sample"])
def test_every_tensor_is_checked(launched, op):  # noqa: F811
    import torch
    kinds = _tensors(torch)[op]
    if op != "pack":
        _call(op, {name: Tensor(*kind) for name, kind in kinds.items()})
        assert len(launched) == 1
    for name, kind in kinds.items():
        for wrong in (Tensor(*kind, at=HOST), Tensor(*kind, at=ELSEWHERE), Tensor(*kind, contiguous=False),
                      Tensor(torch.float64, *kind[1:]), Tensor(*kind[:-1], kind[-1] + 1)):
            if name in ("logits", "workspace") and wrong.shape != kind[1:]:
                continue                                                    # any vocabulary; the library looks at the size
            t = {n: Tensor(*k) for n, k in kinds.items()}
            t[name] = wrong
            for other in t.values():
                other.dim = lambda o=other: len(o.shape)
            with pytest.raises(ValueError):
                _call(op, t)
                pytest.fail(f"{name}: {wrong.device}, {wrong.dtype}, {wrong.shape}, contiguous {wrong.contiguous_}")
    assert len(launched) == (op != "pack")


def test_binding_refuses_shapes(lib):
    import torch
    for n, k, group in ((0, 256, 64), (40, 200, 64), (40, 256, 48)):
        with pytest.raises(ValueError, match="group"):
            tq.PackedQ4(None, None, None, n, k, group)
    with pytest.raises(ValueError, match="codes"):
        tq.pack_q4(torch.zeros(4, 128, dtype=torch.uint8), torch.ones(4, 1).half())


def test_source_hash_leaves_out_these_sources(monkeypatch, tmp_path):
    """The files of the 4-bit products and of sampling are no part of the step kernel, and none of its files includes one."""
    import os

    import bench
    real = os.path.join(bench.ROOT, "ternary_weight_dp4a_gb300", "csrc")
    others = (bench.OTHER_KERNELS_PREFIX, *bench.MORE_KERNELS_PREFIXES)
    for name in os.listdir(real):
        if name.endswith((".cu", ".cuh", ".h")) and not name.startswith(others) and name not in bench.HOST_ONLY_SOURCES:
            text = open(os.path.join(real, name)).read()
            assert not any(f'#include "{prefix}' in text for prefix in bench.MORE_KERNELS_PREFIXES), name
    csrc = tmp_path / "ternary_weight_dp4a_gb300" / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "k.cu").write_text("kernel")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    h0 = bench.source_hash()
    (csrc / "tq_q4_other.cu").write_text("a product")
    (csrc / "tq_sample.cu").write_text("sampling")
    assert bench.source_hash() == h0


@pytest.fixture
def allocations(monkeypatch):
    """Calls that launch nothing, on CPU tensors; the list says of each tensor that they allocate whether it
    was made under the explicit stream."""
    import contextlib
    import types

    import torch
    made, current = [], []

    @contextlib.contextmanager
    def under(stream):
        current.append(stream)
        yield
        current.pop()

    class Library(types.SimpleNamespace):
        def __getattr__(self, name):
            return lambda *a: 1 << 16 if name.endswith("_bytes") else 0

    monkeypatch.setattr(tq, "load", lambda: Library())
    monkeypatch.setattr(tq, "_tensor", lambda *a, **k: 0x1000)
    monkeypatch.setattr(tq, "_device", lambda: -1)                   # where CPU tensors are
    monkeypatch.setattr(torch.cuda, "stream", under)
    for name in ("empty", "zeros"):
        real = getattr(torch, name)

        def make(*a, real=real, **k):
            made.append(bool(current) and isinstance(current[-1], Stream))
            return real(*a, **k)

        monkeypatch.setattr(torch, name, make)
    return made


@pytest.mark.parametrize("call,count", [("pack", 3), ("gemv", 2), ("gateup", 2), ("sample", 2)])
def test_a_call_allocates_on_its_stream(allocations, call, count):
    import torch
    u8, half = torch.full((48 * 128,), 1, dtype=torch.uint8), torch.full((48 * 4,), 1.0).half()
    w = tq.PackedQ4(u8, half, half, 40, 256, 64)
    x = torch.full((20, 256), 1.0).bfloat16()
    calls = {
        "pack": lambda st: tq.pack_q4(torch.full((40, 256), 1, dtype=torch.uint8), torch.full((40, 4), 1.0).half(),
                                      torch.full((40, 4), 1.0).half(), stream=st),
        "gemv": lambda st: tq.q4_gemv(w, x, stream=st),
        "gateup": lambda st: tq.q4_gateup(w, w, x, stream=st),
        "sample": lambda st: tq.sample(torch.full((3, 50), 1.0), torch.full((3,), 0.5), stream=st),
    }
    allocations.clear()
    calls[call](Stream())
    assert len(allocations) == count and all(allocations)


def test_weights_can_be_copied_and_pickled(launched):  # noqa: F811
    import copy
    import pickle

    import torch
    w = tq.PackedQ4(Tensor(torch.uint8, 48 * 128), Tensor(torch.float16, 48 * 4), None, 40, 256, 64)
    for other in (copy.deepcopy(w), copy.copy(w), pickle.loads(pickle.dumps(w))):
        assert (other.n, other.k, other.group, other.mins) == (40, 256, 64, None) and other.nbytes == w.nbytes


def test_what_earlier_work_writes_is_not_read_as_read_only():
    """These kernels start before the work ahead of them in the stream has ended: nothing of theirs is read through
    const __restrict__, __ldg or the read-only path."""
    import glob
    import os
    import re
    seen = 0
    for path in glob.glob(os.path.join(os.path.dirname(tq.__file__), "csrc", "tq_q4_*.cu")) + \
            glob.glob(os.path.join(os.path.dirname(tq.__file__), "csrc", "tq_sample.cu")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        seen += 1
        assert "__restrict__" not in text and "__ldg" not in text and ".nc" not in text, path
    assert seen == 5


def test_workspace_of_the_most_rows_does_for_fewer(lib):
    for group in (32, 64, 128):
        sizes = [lib.tq_q4_workspace_bytes(m, 1024, group) for m in range(1, 1200)]
        assert sizes == sorted(sizes) and sizes[15] == 0 and sizes[16] > 0
    # parts of the sums: 32 bf16 for every row and 128 values; sums: fp32 for every group and 16 rows at a time
    assert lib.tq_q4_workspace_bytes(512, 1024, 32) == 512 * 8 * 64 and lib.tq_q4_workspace_bytes(100, 1024, 128) == 112 * 8 * 4
