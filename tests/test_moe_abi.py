"""The mixture-of-experts entry points reject bad arguments before touching the
GPU, size their workspace as documented, and the binding refuses tensors that
the kernels could not read.  No GPU needed."""
import ctypes

import pytest

from ternary_weight_dp4a_gb300 import build as tqbuild
from ternary_weight_dp4a_gb300 import tq

OK, ARG, ALIGN, WS = 0, 1, 2, 4
ST = ctypes.c_void_p(0)


def P(a):
    return ctypes.c_void_p(a)


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    return tq.load()


def _x(codes=0x1000, scales=0x2000, experts=4, n=256, k=256, fmt=0):
    return tq._Experts(codes, scales, experts, n, k, fmt)


def _up256(v):
    return (v + 255) // 256 * 256


def test_workspace_bytes(lib):
    m, topk, e, h, i = 3, 2, 4, 256, 512
    slots = m * topk
    want = 256 + _up256(slots * (2 * max(h, i) + 16)) + _up256(e * 4) + _up256((e + 1) * 4) + 2 * _up256(slots * 4) \
        + _up256(slots * i * 2) + _up256(slots * i) + _up256(slots * (i // 128) * 4) + _up256(slots * h * 4)
    assert lib.tq_moe_workspace_bytes(m, topk, e, h, i) == want
    assert lib.tq_moe_workspace_bytes(m, topk, e, 0, 0) > 0                 # for the plan alone
    for bad in ((0, 2, 4, h, i), (3, 0, 4, h, i), (3, 5, 4, h, i), (3, 2, 0, h, i), (3, 2, 1025, h, i), (3, 33, 64, h, i),
                (3, 2, 4, 200, i), (3, 2, 4, h, 0), (3, 2, 4, 65536, i), (1 << 26, 2, 4, h, i)):
        assert lib.tq_moe_workspace_bytes(*bad) == 0, bad


def test_norm_rejects(lib):
    def call(res=0x1000, rt=0, delta=0x2000, dt=1, gamma=0x3000, m=2, n=256, eps=1e-6, out=0x4000, x=0x5000, q=0x6000,
             s=0x7000):
        return lib.tq_add_rmsnorm_rotq(P(res), rt, P(delta), dt, P(gamma), m, n, ctypes.c_float(eps), P(out), P(x), P(q),
                                       P(s), ST)
    assert call(res=0) == ARG and call(m=0) == ARG and call(rt=2) == ARG and call(dt=-1) == ARG
    assert call(n=100) == ARG and call(n=0) == ARG and call(n=32768 + 128) == ARG
    assert call(q=0) == ARG and call(s=0) == ARG                            # one without the other
    assert call(q=0, s=0, x=0, out=0) == ARG                                # no output
    assert call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG
    for name in ("res", "delta", "gamma", "out", "x", "q"):
        assert call(**{name: 0x8008}) == ALIGN, name
    assert call(s=0x7002) == ALIGN


def test_route_and_plan_reject(lib):
    def route(l=0x1000, lt=0, m=2, e=8, k=2, ids=0x2000, w=0x3000):
        return lib.tq_moe_route(P(l), lt, m, e, k, 1, P(ids), P(w), ST)
    assert route(l=0) == ARG and route(ids=0) == ARG and route(w=0) == ARG and route(lt=3) == ARG
    assert route(m=0) == ARG and route(e=0) == ARG and route(e=1025, k=2) == ARG and route(k=9) == ARG and route(k=0) == ARG
    assert route(e=64, k=33) == ARG and route(m=1 << 26) == ARG
    assert route(l=0x1002) == ALIGN and route(ids=0x2001) == ALIGN

    need = lib.tq_moe_workspace_bytes(2, 2, 8, 0, 0)

    def plan(ids=0x1000, m=2, k=2, e=8, off=0x2000, rows=0x3000, pos=0x4000, ws=0x10000, wsb=need):
        return lib.tq_moe_plan(P(ids), m, k, e, P(off), P(rows), P(pos), P(ws), wsb, ST)
    assert plan(ids=0) == ARG and plan(off=0) == ARG and plan(rows=0) == ARG and plan(pos=0) == ARG
    assert plan(m=0) == ARG and plan(k=9) == ARG and plan(e=2000) == ARG
    assert plan(off=0x2002) == ALIGN and plan(ws=0x10010) == ALIGN
    assert plan(ws=0) == ARG and plan(wsb=need - 1) == WS


def test_products_reject(lib):
    need = 256 + 6 * (2 * 256 + 16)

    def gemv(w=_x(), q=0x3000, s=0x4000, m=3, rows=0x5000, off=0x6000, slots=6, y=0x7000, ws=0x10000, wsb=need):
        return lib.tq_moe_gemv(ctypes.byref(w) if w else None, P(q), P(s), m, P(rows), P(off), slots, P(y), P(ws), wsb, ST)
    assert gemv(w=None) == ARG
    for bad in (dict(codes=0), dict(scales=0), dict(experts=0), dict(experts=1025), dict(n=0), dict(n=32769), dict(k=100),
                dict(k=0), dict(k=32768 + 128), dict(fmt=2)):
        assert gemv(w=_x(**bad)) == ARG, bad
    assert gemv(w=_x(codes=0x1010)) == ALIGN and gemv(w=_x(scales=0x2001)) == ALIGN
    assert gemv(q=0) == ARG and gemv(s=0) == ARG and gemv(off=0) == ARG and gemv(y=0) == ARG
    assert gemv(m=0) == ARG and gemv(slots=0) == ARG and gemv(slots=(1 << 26) + 1) == ARG
    assert gemv(rows=0, slots=4) == ARG                                     # more slots than rows of q
    assert gemv(q=0x3008) == ALIGN and gemv(s=0x4002) == ALIGN and gemv(rows=0x5002) == ALIGN and gemv(y=0x7002) == ALIGN
    assert gemv(ws=0) == ARG and gemv(ws=0x10010) == ALIGN and gemv(wsb=need - 1) == WS

    def gateup(g=_x(), u=_x(), h=0x7000, wsb=need):
        return lib.tq_moe_gateup(ctypes.byref(g), ctypes.byref(u), P(0x3000), P(0x4000), 3, P(0x5000), P(0x6000), 6, P(h),
                                 P(0x10000), wsb, ST)
    for bad in (dict(n=128), dict(k=128), dict(fmt=1), dict(experts=2)):
        assert gateup(u=_x(**bad)) == ARG, bad
    assert gateup(h=0) == ARG and gateup(h=0x7001) == ALIGN and gateup(wsb=need - 1) == WS


def test_combine_and_ffn_reject(lib):
    def combine(y=0x1000, pos=0x2000, w=0x3000, m=2, k=2, slots=4, n=256, out=0x4000, ot=0):
        return lib.tq_moe_combine(P(y), P(pos), P(w), m, k, slots, n, P(out), ot, ST)
    assert combine(y=0) == ARG and combine(pos=0) == ARG and combine(w=0) == ARG and combine(out=0) == ARG
    assert combine(m=0) == ARG and combine(k=0) == ARG and combine(k=33) == ARG and combine(slots=0) == ARG
    assert combine(n=6) == ARG and combine(n=0) == ARG and combine(ot=2) == ARG
    assert combine(y=0x1004) == ALIGN and combine(out=0x4008) == ALIGN and combine(w=0x3002) == ALIGN

    need = lib.tq_moe_workspace_bytes(2, 2, 4, 256, 512)

    def ffn(g=_x(n=512), u=_x(n=512), d=_x(n=256, k=512), q=0x3000, s=0x4000, ids=0x5000, w=0x6000, m=2, k=2, out=0x7000,
            ot=1, ws=0x10000, wsb=need):
        return lib.tq_moe_ffn(ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), P(q), P(s), P(ids), P(w), m, k, P(out), ot,
                              P(ws), wsb, ST)
    assert ffn(d=_x(n=256, k=256)) == ARG and ffn(d=_x(n=128, k=512)) == ARG and ffn(d=_x(n=256, k=512, fmt=1)) == ARG
    assert ffn(d=_x(n=256, k=512, experts=3)) == ARG and ffn(u=_x(n=256)) == ARG
    assert ffn(g=_x(n=500), u=_x(n=500), d=_x(n=256, k=512)) == ARG         # inter not a multiple of 128
    assert ffn(q=0) == ARG and ffn(ids=0) == ARG and ffn(w=0) == ARG and ffn(out=0) == ARG and ffn(ot=5) == ARG
    assert ffn(m=0) == ARG and ffn(k=5) == ARG
    assert ffn(q=0x3004) == ALIGN and ffn(out=0x7004) == ALIGN
    assert ffn(ws=0) == ARG and ffn(ws=0x10020) == ALIGN and ffn(wsb=need - 1) == WS


def test_binding_refuses_tensors_the_kernels_cannot_read(lib):
    import torch
    x = torch.zeros(2, 256)
    with pytest.raises(ValueError, match="residual"):
        tq.add_rmsnorm_rotq(x)                                              # not on a GPU
    with pytest.raises(ValueError, match="logits"):
        tq.moe_route(x, 2)
    with pytest.raises(ValueError, match="ids"):
        tq.moe_plan(torch.zeros(2, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="codes"):
        tq.PackedExperts(torch.zeros(4, 8, 64, dtype=torch.uint8), torch.zeros(4, 8, 2).half(), 4, 8, 256, 0)
    with pytest.raises(ValueError, match="out of range"):
        tq.moe_workspace(1, 9, 8)
