"""The mixture-of-experts calls of the binding refuse a tensor that is not on the device where
they launch, of another type or not contiguous, before anything is launched.  The tensors here
only say where they are; the library only notes that it was called.  No GPU needed."""
import copy
import math
import pickle

import pytest

from ternary_weight_dp4a_gb300 import tq

HERE, ELSEWHERE, HOST = 0, 1, -1


class Tensor:
    def __init__(self, dtype, *shape, at=HERE, contiguous=True):
        self.dtype, self.shape, self.at, self.contiguous_ = dtype, shape, at, contiguous

    device = property(lambda self: "cpu" if self.at < 0 else f"cuda:{self.at}")
    is_cuda = property(lambda self: self.at >= 0)

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return self.contiguous_

    def stride(self):
        return self.shape

    def numel(self):
        return math.prod(self.shape)

    def data_ptr(self):
        return 0x1000


class Stream:
    cuda_stream = 0


@pytest.fixture
def launched(monkeypatch):
    """The names of the library's functions that were called; CUDA as on a box with two devices."""
    names = []

    class Library:
        def __getattr__(self, name):
            def call(*a):
                if name.endswith("_bytes"):
                    return 4096
                names.append(name)
                return 0
            return call

    monkeypatch.setattr(tq, "load", lambda: Library())
    monkeypatch.setattr(tq, "_device", lambda: HERE, raising=False)
    return names


M, TOPK, E, H, I = 3, 2, 4, 256, 128


def _tensors(torch):
    u8, i8, i32, f32, f16, bf16 = torch.uint8, torch.int8, torch.int32, torch.float32, torch.float16, torch.bfloat16
    return {
        "norm": dict(residual=(bf16, M, H), delta=(f32, M, H), gamma=(bf16, H), residual_out=(bf16, M, H), x_out=(bf16, M, H),
                     q=(i8, M, H), s=(f32, M, H // 128)),
        "route": dict(logits=(f32, M, E), ids=(i32, M, TOPK), weights=(f32, M, TOPK)),
        "plan": dict(ids=(i32, M, TOPK), offsets=(i32, E + 1), rows=(i32, M * TOPK), pos=(i32, M, TOPK), workspace=(u8, 4096)),
        "gemv": dict(codes=(u8, E, I, H // 4), scales=(f16, E, I, H // 128), q=(i8, M, H), s=(f32, M, H // 128),
                     offsets=(i32, E + 1), rows=(i32, M * TOPK), y=(f32, M * TOPK, I), workspace=(u8, 4096)),
        "gateup": dict(codes=(u8, E, I, H // 4), scales=(f16, E, I, H // 128), codes2=(u8, E, I, H // 4),
                       scales2=(f16, E, I, H // 128), q=(i8, M, H), s=(f32, M, H // 128), offsets=(i32, E + 1),
                       rows=(i32, M * TOPK), h=(bf16, M * TOPK, I), workspace=(u8, 4096)),
        "combine": dict(y=(f32, M * TOPK, H), pos=(i32, M, TOPK), weights=(f32, M, TOPK), out=(bf16, M, H)),
        "ffn": dict(codes=(u8, E, I, H // 4), scales=(f16, E, I, H // 128), codes2=(u8, E, I, H // 4),
                    scales2=(f16, E, I, H // 128), codes3=(u8, E, H, I // 4), scales3=(f16, E, H, I // 128), q=(i8, M, H),
                    s=(f32, M, H // 128), ids=(i32, M, TOPK), weights=(f32, M, TOPK), out=(f32, M, H), workspace=(u8, 4096)),
    }


def _call(op, t):
    x = lambda c="codes", s="scales", n=I, k=H: tq.PackedExperts(t[c], t[s], E, n, k, 0)  # noqa: E731
    plan = lambda: tq.MoePlan(t.get("offsets"), t.get("rows"), t.get("pos"))  # noqa: E731
    st = Stream()
    if op == "norm":
        return tq.add_rmsnorm_rotq(t["residual"], t["delta"], t["gamma"], residual_out=t["residual_out"], x_out=t["x_out"],
                                   q=t["q"], s=t["s"], stream=st)
    if op == "route":
        return tq.moe_route(t["logits"], TOPK, ids=t["ids"], weights=t["weights"], stream=st)
    if op == "plan":
        return tq.moe_plan(t["ids"], E, plan=plan(), workspace=t["workspace"], stream=st)
    if op == "gemv":
        return tq.moe_gemv(x(), t["q"], t["s"], plan(), gather=True, y=t["y"], workspace=t["workspace"], stream=st)
    if op == "gateup":
        return tq.moe_gateup(x(), x("codes2", "scales2"), t["q"], t["s"], plan(), h=t["h"], workspace=t["workspace"], stream=st)
    if op == "combine":
        return tq.moe_combine(t["y"], tq.MoePlan(None, None, t["pos"]), t["weights"], out=t["out"], stream=st)
    return tq.moe_ffn(x(), x("codes2", "scales2"), x("codes3", "scales3", H, I), t["q"], t["s"], t["ids"], t["weights"],
                      out=t["out"], workspace=t["workspace"], stream=st)


OPS = ("norm", "route", "plan", "gemv", "gateup", "combine", "ffn")


@pytest.mark.parametrize("op", OPS)
def test_every_tensor_is_checked(launched, op):
    import torch
    kinds = _tensors(torch)[op]
    _call(op, {name: Tensor(*kind) for name, kind in kinds.items()})
    assert len(launched) == 1
    for name, kind in kinds.items():
        for wrong in (Tensor(*kind, at=HOST), Tensor(*kind, at=ELSEWHERE), Tensor(*kind, contiguous=False),
                      Tensor(torch.float64, *kind[1:])):
            t = {n: Tensor(*k) for n, k in kinds.items()}
            t[name] = wrong
            with pytest.raises(ValueError):
                _call(op, t)
                pytest.fail(f"{name}: {wrong.device}, {wrong.dtype}, contiguous {wrong.contiguous_}")
    assert len(launched) == 1


def test_weights_can_be_copied_and_pickled(launched):
    """As PackedWeight's; and a call takes the addresses that its tensors have then."""
    import torch
    w = tq.PackedExperts(Tensor(torch.uint8, E, I, H // 4), Tensor(torch.float16, E, I, H // 128), E, I, H, 0)
    for other in (copy.deepcopy(w), copy.copy(w), pickle.loads(pickle.dumps(w))):
        assert (other.experts, other.n, other.k, other.fmt) == (E, I, H, 0) and other.codes.shape == w.codes.shape
    w.codes.data_ptr = lambda: 0x2000
    assert w.c_struct().codes == 0x2000 and w.c_struct().scales == 0x1000


def test_the_library_keeps_the_bits_of_lost_waits(monkeypatch):
    """A call without a workspace drops the one that it took; its waits are still to be seen."""
    from ternary_weight_dp4a_gb300 import build
    build.build()
    assert tq.load().tq_moe_read_error_word(None, 0) == 1                   # nowhere to put them

    class Library:
        def tq_moe_read_error_word(self, value, stream):
            value._obj.value = 1 << 12
            return tq.TQ_ERR_TIMEOUT

        def tq_status_string(self, status):
            return b"timeout"

        def tq_last_cuda_error(self):
            return 0

    monkeypatch.setattr(tq, "load", lambda: Library())
    with pytest.raises(tq.TQError) as e:
        tq.moe_read_error_word(Stream())
    assert e.value.status == tq.TQ_ERR_TIMEOUT
