"""Calls with an explicit stream: what they allocate for themselves belongs to that stream."""
import contextlib
import types

import pytest

from ternary_weight_dp4a_gb300 import tq


class Stream:
    cuda_stream = 7


@pytest.fixture
def allocations(monkeypatch):
    """Calls that launch nothing, on CPU tensors; the list says of each tensor that they allocate
    whether it was made under the explicit stream."""
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
    for name in ("empty", "empty_like", "zeros"):
        real = getattr(torch, name)

        def make(*a, real=real, **k):
            made.append(bool(current) and isinstance(current[-1], Stream))
            return real(*a, **k)

        monkeypatch.setattr(torch, name, make)
    return made


def _experts(torch, experts, n, k):
    return tq.PackedExperts(torch.ones((experts, n, k // 4), dtype=torch.uint8), torch.ones((experts, n, k // 128)).half(),
                            experts, n, k, 0)


def _calls(torch):
    m, topk, e, h, i = 3, 2, 4, 256, 128
    q, s = torch.ones((m, h), dtype=torch.int8), torch.ones((m, h // 128))
    ids, w = torch.ones((m, topk), dtype=torch.int32), torch.ones((m, topk))
    plan = tq.MoePlan(torch.ones(e + 1, dtype=torch.int32), torch.ones(m * topk, dtype=torch.int32), ids)
    gate, up, down = _experts(torch, e, i, h), _experts(torch, e, i, h), _experts(torch, e, h, i)
    return {
        "norm": lambda st: tq.add_rmsnorm_rotq(torch.ones((m, h)), stream=st),
        "route": lambda st: tq.moe_route(torch.ones((m, e)), topk, stream=st),
        "plan": lambda st: tq.moe_plan(ids, e, stream=st),
        "gemv": lambda st: tq.moe_gemv(gate, q, s, plan, gather=True, stream=st),
        "gateup": lambda st: tq.moe_gateup(gate, up, q, s, plan, stream=st),
        "combine": lambda st: tq.moe_combine(torch.ones((m * topk, h)), plan, w, stream=st),
        "ffn": lambda st: tq.moe_ffn(gate, up, down, q, s, ids, w, stream=st),
        "pack": lambda st: tq.pack_experts(torch.ones((e, i, h), dtype=torch.uint8), 0, torch.ones((e, i, h // 128)).half(),
                                           stream=st),
        "rotq": lambda st: tq.rotate_quant(torch.ones((m, h)).bfloat16(), stream=st),
        "dense": lambda st: tq.gemv(tq.PackedWeight(gate.codes[0], gate.scales[0], i, h, 0), q, s, stream=st),
    }


@pytest.mark.parametrize("call", ["norm", "route", "plan", "gemv", "gateup", "combine", "ffn", "pack", "rotq", "dense"])
def test_a_call_allocates_on_its_stream(allocations, call):
    import torch
    calls = _calls(torch)
    allocations.clear()
    calls[call](Stream())
    assert allocations and all(allocations)


@pytest.mark.parametrize("call", ["plan", "gemv", "gateup", "ffn"])
def test_a_call_fills_no_more_than_the_error_word(allocations, monkeypatch, call):
    """Without a workspace a call takes one for itself; a fill of all of it would cost more than the call."""
    import torch
    filled = []
    for owner, name in ((torch, "zeros"), (torch, "full"), (torch.Tensor, "zero_"), (torch.Tensor, "fill_")):
        real = getattr(owner, name)

        def fill(*a, real=real, **k):
            out = real(*a, **k)
            filled.append(out.numel() * out.element_size())
            return out

        monkeypatch.setattr(owner, name, fill)
    calls = _calls(torch)
    filled.clear()
    calls[call](Stream())
    assert sum(filled) <= 256


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_calls_beside_a_busy_current_stream(handle):
    """The current stream is held up while a layer runs on another one, and then takes memory:
    neither what it still has to do nor what it takes may reach the layer's buffers."""
    import torch
    experts, topk, hidden, inter, m = 8, 2, 512, 256, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    gate, up, down = (tq.pack_experts(torch.randint(0, 3, (experts, n, k), generator=gen, device="cuda", dtype=torch.uint8), 0,
                                      (0.01 + 0.04 * torch.rand((experts, n, k // 128), generator=gen, device="cuda")).half())
                      for n, k in ((inter, hidden), (inter, hidden), (hidden, inter)))
    x = torch.randn((m, hidden), generator=gen, device="cuda")
    logits = torch.randn((m, experts), generator=gen, device="cuda")

    def layer(**stream):
        _, q, s = tq.add_rmsnorm_rotq(x, **stream)
        ids, w = tq.moe_route(logits, topk, **stream)
        y = tq.moe_ffn(gate, up, down, q, s, ids, w, **stream)
        plan = tq.moe_plan(ids, experts, **stream)
        h = tq.moe_gateup(gate, up, q, s, plan, **stream)
        return y, h, tq.moe_gemv(gate, q, s, plan, gather=True, **stream)

    want = layer()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                                   # 50 ms of the current stream
    got = layer(stream=side.cuda_stream if handle else side)
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                               # and of the other one
    got = layer(stream=side.cuda_stream if handle else side)
    taken = [torch.full((1 << 20,), 85, dtype=torch.uint8, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert len(taken) == 16
    for a, b in zip(got, want):
        assert torch.equal(a, b)
