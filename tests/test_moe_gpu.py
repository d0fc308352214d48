"""The mixture-of-experts layer on the GPU against plain implementations in 64
bits (numpy), at the sizes and routings where it can go wrong.

Tolerances, from the roundings each formula has (u = 2^-24, half a step of fp32):
  products   fold of nb fused multiply-adds over terms t_b, each scale product
             rounded once:  |y - y64| <= (nb + 1) u sum|t_b|  (first order; times 1.01)
  gate/up    bf16 rounding 2^-8 |h|, plus the fp32 errors of g and u carried
             through SiLU (slope <= 1.1) and 8 u of its own steps
  weights    expf within 2 ulp, its argument within u |l - l0|, both in the
             numerator and the sum, 6 additions and a division
  sum        topk fused multiply-adds: topk u sum|w y|, and half a step of bf16
Codes, scales, ids and the plan are exact.
"""
import numpy as np
import pytest

from _util import bf16_tensor
from ternary_weight_dp4a_gb300 import synth

pytestmark = pytest.mark.gpu
B = 128
U = 2.0 ** -24


@pytest.fixture(scope="module")
def tq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ternary_weight_dp4a_gb300 import build, tq as tqmod
    build.build()
    tqmod.load()
    return tqmod


# ----------------------------------------------------------------------------
# plain implementations
# ----------------------------------------------------------------------------

def bf16_round(x32):
    """fp32 -> bf16 (to nearest, ties to even), as fp32."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x32, np.float32)).to(torch.bfloat16).float().numpy()


def bf16_bits_of(x32):
    return (np.ascontiguousarray(x32, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def norm_ref(orc, residual, delta, gamma, eps, res_bf16):
    t = residual if delta is None else (residual + delta).astype(np.float32)
    if res_bf16:
        t = bf16_round(t)
    t64 = t.astype(np.float64)
    with np.errstate(divide="ignore"):
        inv = (1.0 / np.sqrt((t64 * t64).sum(1) / t.shape[1] + float(np.float32(eps)))).astype(np.float32)
    with np.errstate(invalid="ignore"):
        x = t * inv[:, None]
        if gamma is not None:
            x = x * gamma[None, :]
    x = bf16_round(x)
    q, s = orc.rotate_quant(bf16_bits_of(x))
    return t, x, q, s


class Experts:
    def __init__(self, tq, experts, n, k, fmt, seed):
        import torch
        mats = [synth.weight(n, k, fmt, seed + e) for e in range(experts)]
        self.codes, self.scales = np.stack([c for c, _ in mats]), np.stack([s for _, s in mats])
        self.n, self.k, self.fmt = n, k, fmt
        self.dev = tq.pack_experts(torch.from_numpy(self.codes).cuda(), fmt, torch.from_numpy(self.scales).cuda())

    def terms(self, e, q, s):
        """Block terms d_b * scale_w * scale_a in 64 bits, [rows][n][nb]."""
        c = self.codes[e].astype(np.int64)
        w = np.where(c == 2, -1, c) if self.fmt == 0 else 2 * c - 1
        nb = self.k // B
        d = np.einsum("nbj,rbj->rnb", w.reshape(self.n, nb, B), q.astype(np.int64).reshape(len(q), nb, B))
        return d * self.scales[e].astype(np.float64)[None] * s.astype(np.float64)[:, None, :]


def act(m, k, seed=7):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k // B, B))
    s = (np.abs(x).max(2) / 127).astype(np.float32)
    q = np.clip(np.rint(x / s[..., None]), -127, 127).astype(np.int8)
    return q.reshape(m, k), s


def plan_ref(ids, experts):
    flat = ids.reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < experts)
    key = np.where(ok, flat, experts)
    order = np.argsort(key, kind="stable")
    total = int(ok.sum())
    offsets = np.searchsorted(key[order], np.arange(experts + 1))
    rows = np.full(flat.size, -1)
    rows[:total] = order[:total] // ids.shape[1]
    pos = np.full(flat.size, -1)
    pos[order[:total]] = np.arange(total)
    return offsets.astype(np.int32), rows.astype(np.int32), pos.astype(np.int32).reshape(ids.shape)


def ragged_ids(counts, topk=1, seed=0, dropped=0):
    """ids [m][topk] in which expert e occurs counts[e] times, plus `dropped` slots without one."""
    rng = np.random.default_rng(seed)
    flat = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(dropped, -1)])
    flat = np.concatenate([flat, np.full(-len(flat) % topk, -1)])
    return rng.permutation(flat).astype(np.int32).reshape(-1, topk)


def cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(t):
    import torch
    return t.contiguous().view({2: torch.int16, 4: torch.int32, 1: torch.int8}[t.element_size()]).cpu().numpy()


# ----------------------------------------------------------------------------
# norm
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("res,delta,gamma", [("f32", "f32", True), ("f32", "bf16", False), ("bf16", "bf16", True),
                                             ("bf16", "f32", False), ("bf16", None, True), ("f32", None, False)])
@pytest.mark.parametrize("m,n", [(1, 128), (3, 384), (2, 5120), (5, 1152), (1, 32768), (700, 256)])
def test_add_rmsnorm_rotq_bit_exact(tq, orc, m, n, res, delta, gamma):
    import torch
    rng = np.random.default_rng(m * n)
    r = (4 * rng.standard_normal((m, n))).astype(np.float32)
    d = None if delta is None else rng.standard_normal((m, n)).astype(np.float32)
    g = bf16_round(1 + 0.2 * rng.standard_normal(n)) if gamma else None
    r = bf16_round(r) if res == "bf16" else r
    d = bf16_round(d) if delta == "bf16" else d
    if m >= 3:
        r[1] = 0                                   # a row of zeros
        r[2] *= 1e-3
        if d is not None:
            d[1] = 0
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    rd = cuda(r).to(dt[res])
    x_out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    out, q, s = tq.add_rmsnorm_rotq(rd, None if d is None else cuda(d).to(dt[delta]),
                                    None if g is None else cuda(g).to(torch.bfloat16), eps=1e-5, x_out=x_out)
    r = rd.float().cpu().numpy()                   # as the call got it
    t_ref, x_ref, q_ref, s_ref = norm_ref(orc, r, d, g, 1e-5, res == "bf16")
    assert np.array_equal(out.float().cpu().numpy(), t_ref)
    assert np.array_equal(x_out.float().cpu().numpy(), x_ref)
    assert np.array_equal(q.cpu().numpy(), q_ref)
    assert np.array_equal(bits(s), s_ref.view(np.int32))
    # in place, and without the optional outputs
    out2, q2, s2 = tq.add_rmsnorm_rotq(rd, None if d is None else cuda(d).to(dt[delta]),
                                       None if g is None else cuda(g).to(torch.bfloat16), eps=1e-5, residual_out=rd)
    assert out2 is rd and torch.equal(rd, out) and torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("scale", [1e20, 1e-20, 3e38])
def test_norm_of_values_whose_squares_leave_binary32(tq, orc, scale):
    rng = np.random.default_rng(3)
    r = np.clip(scale * rng.standard_normal((2, 256)), -3.3e38, 3.3e38).astype(np.float32)
    _, q, s = tq.add_rmsnorm_rotq(cuda(r), eps=0.0)
    _, _, q_ref, s_ref = norm_ref(orc, r, None, None, 0.0, False)
    assert np.array_equal(q.cpu().numpy(), q_ref) and np.array_equal(bits(s), s_ref.view(np.int32))


def test_norm_nan_stays_in_its_row(tq, orc):
    rng = np.random.default_rng(4)
    r = rng.standard_normal((4, 512)).astype(np.float32)
    r[1, 5], r[2, 300] = np.nan, np.inf
    _, q, s = tq.add_rmsnorm_rotq(cuda(r))
    _, _, q_ref, s_ref = norm_ref(orc, r[[0, 3]], None, None, 1e-6, False)
    assert np.array_equal(q.cpu().numpy()[[0, 3]], q_ref) and np.array_equal(bits(s)[[0, 3]], s_ref.view(np.int32))
    s = s.cpu().numpy()
    assert np.isnan(s[1]).all() and np.isnan(s[2, 2]) and (s[2, [0, 1, 3]] == 0).all()
    assert (q.cpu().numpy()[1] == 0).all()


# ----------------------------------------------------------------------------
# router and plan
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("m,experts,topk,bf16", [(1, 1, 1, False), (3, 7, 7, False), (9, 64, 8, True), (33, 65, 6, True),
                                                 (17, 256, 8, True), (5, 1000, 32, False), (2, 1024, 4, True)])
def test_route(tq, m, experts, topk, bf16, renorm):
    import torch
    rng = np.random.default_rng(m + experts)
    l = rng.standard_normal((m, experts)).astype(np.float32) * 2
    l = bf16_round(np.round(l * 4) / 4) if bf16 else l                # many ties
    if m >= 3 and experts > 2:
        l[0] = -np.inf                                                # nothing to choose
        l[1, 1:] = -np.inf                                            # one choice
        l[1, 0] = np.inf
        l[2, :2] = [np.nan, -0.0]
    lt = cuda(l).to(torch.bfloat16) if bf16 else cuda(l)
    ids, w = tq.moe_route(lt, topk, renormalize=renorm)
    v = np.where(np.isnan(l), -np.inf, l).astype(np.float64)
    v = np.minimum(v, float(np.finfo(np.float32).max))
    order = np.argsort(-v, axis=1, kind="stable")[:, :topk]
    top = np.take_along_axis(v, order, 1)
    none = top == -np.inf
    assert np.array_equal(ids.cpu().numpy(), np.where(none, -1, order))
    l0 = np.where(none[:, :1], 0, top[:, :1])
    e = np.exp(top - l0)
    total = np.where(renorm, e.sum(1), np.exp(v - l0).sum(1))
    ref = np.where(none, 0, e / np.where(total == 0, 1, total)[:, None])
    gap = np.where(none, 0, np.abs(top - l0))
    terms = topk if renorm else experts
    rel = (2 * (4 + np.minimum(gap.max(1, keepdims=True), 100)) + terms + 2) * U
    assert (np.abs(w.cpu().numpy() - ref) <= rel * ref + 1e-37).all()


@pytest.mark.parametrize("m,topk,experts", [(1, 1, 1), (1, 8, 64), (33, 6, 64), (1024, 1, 3), (1025, 1, 1024), (700, 8, 256),
                                            (5000, 4, 17)])
def test_plan(tq, m, topk, experts):
    rng = np.random.default_rng(m)
    ids = rng.integers(-1, experts + 1, (m, topk)).astype(np.int32)   # -1 and `experts` have no expert
    ids[rng.random((m, topk)) < 0.3] = experts // 2                   # one popular expert, repeated in a token
    plan = tq.moe_plan(cuda(ids), experts)
    offsets, rows, pos = plan_ref(ids, experts)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.rows.cpu().numpy().ravel(), rows)
    assert np.array_equal(plan.pos.cpu().numpy(), pos)


def test_plan_with_no_expert_at_all(tq):
    ids = np.full((3, 4), -1, np.int32)
    plan = tq.moe_plan(cuda(ids), 9)
    assert (plan.offsets.cpu().numpy() == 0).all() and (plan.rows.cpu().numpy() == -1).all()
    assert (plan.pos.cpu().numpy() == -1).all()


# ----------------------------------------------------------------------------
# products
# ----------------------------------------------------------------------------

# rows per expert: none, one, around the 8-row and 16-row chunks, and on both sides of
# the tile kernel's first row and of its one, two and three tiles
COUNTS = [[1], [0, 0, 3], [8, 0, 1, 9], [7, 17, 0, 2, 33], [0, 130, 5], [64, 225, 65, 0, 449, 224],
          [48, 193, 49, 385], [32, 33, 192, 31], [0, 290, 5, 0]]
SHAPES = [(1, 128), (96, 256), (130, 384), (256, 1152), (100, 5120)]


def _product_case(counts, k, topk=2, dropped=1, seed=0):
    ids = ragged_ids(counts, topk, seed, dropped)
    offsets, rows, pos = plan_ref(ids, len(counts))
    q, s = act(ids.shape[0], k, seed + 1)
    return ids, offsets, rows, pos, q, s


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
def test_moe_gemv(tq, counts, n, k, fmt):
    import torch
    ids, offsets, rows, pos, q, s = _product_case(counts, k)
    w = Experts(tq, len(counts), n, k, fmt, seed=11)
    plan = tq.MoePlan(cuda(offsets), cuda(rows), cuda(pos))
    y = torch.full((rows.size, n), np.nan, device="cuda")
    tq.moe_gemv(w.dev, cuda(q), cuda(s), plan, gather=True, y=y)
    got = y.cpu().numpy().astype(np.float64)
    total = offsets[-1]
    assert np.isnan(got[total:]).all()                                # rows behind the plan are not touched
    for e in range(len(counts)):
        at = slice(offsets[e], offsets[e + 1])
        t = w.terms(e, q[rows[at]], s[rows[at]])
        assert (np.abs(got[at] - t.sum(2)) <= 1.01 * (k // B + 1) * U * np.abs(t).sum(2) + 1e-44).all()
    # the rows given in sorted order instead of gathered: the same bits
    r = np.maximum(rows, 0)
    y2 = tq.moe_gemv(w.dev, cuda(q[r]), cuda(s[r]), plan)
    assert np.array_equal(bits(y2)[:total], bits(y)[:total])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,k", [(1, 128), (72, 256), (128, 1152), (200, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
def test_moe_gateup(tq, counts, n, k, fmt):
    import torch
    ids, offsets, rows, pos, q, s = _product_case(counts, k, seed=5)
    g, u = (Experts(tq, len(counts), n, k, fmt, seed=sd) for sd in (20, 90))
    plan = tq.MoePlan(cuda(offsets), cuda(rows), cuda(pos))
    h = torch.full((rows.size, n), np.nan, device="cuda", dtype=torch.bfloat16)
    tq.moe_gateup(g.dev, u.dev, cuda(q), cuda(s), plan, h=h)
    got = h.float().cpu().numpy().astype(np.float64)
    total = offsets[-1]
    assert np.isnan(got[total:]).all()
    nb = k // B
    for e in range(len(counts)):
        at = slice(offsets[e], offsets[e + 1])
        tg, tu = (w.terms(e, q[rows[at]], s[rows[at]]) for w in (g, u))
        g64, u64 = tg.sum(2), tu.sum(2)
        dg, du = (1.01 * (nb + 1) * U * np.abs(t).sum(2) for t in (tg, tu))
        sil = g64 / (1 + np.exp(-g64))
        ref = sil * u64
        tol = (2.0 ** -8 + 8 * U) * np.abs(ref) + 1.01 * (1.1 * dg * np.abs(u64) + np.abs(sil) * du + 1.1 * dg * du) + 1e-38
        assert (np.abs(got[at] - ref) <= tol).all()


def test_product_exact_on_large_codes(tq):
    """Codes +-127 against weights of one sign: the largest block dots, and equal scales of
    one, give whole numbers that every fp32 step holds exactly."""
    import torch
    n, k = 64, 1024
    for fmt, one, minus in ((0, 1, 2), (1, 1, 0)):
        codes = np.full((2, n, k), one, np.uint8)
        codes[1] = minus
        codes[1, 1::2, ::3] = one
        w = tq.pack_experts(cuda(codes), fmt, torch.ones((2, n, k // B), dtype=torch.float16, device="cuda"))
        rng = np.random.default_rng(0)
        q = rng.integers(-127, 128, (6, k)).astype(np.int8)
        q[0], q[1], q[2] = 127, -127, np.arange(k) % 255 - 127
        offsets = np.array([0, 3, 6], np.int32)
        plan = tq.MoePlan(cuda(offsets), cuda(np.arange(6, dtype=np.int32)), cuda(np.arange(6, dtype=np.int32)))
        y = tq.moe_gemv(w, cuda(q), torch.ones((6, k // B), device="cuda"), plan)
        c = codes.astype(np.int64)
        wt = np.where(c == 2, -1, c) if fmt == 0 else 2 * c - 1
        ref = np.concatenate([q[:3].astype(np.int64) @ wt[0].T, q[3:].astype(np.int64) @ wt[1].T])
        assert np.array_equal(y.cpu().numpy(), ref.astype(np.float32))


@pytest.mark.parametrize("fmt", [0, 1])
def test_rows_do_not_depend_on_their_company(tq, fmt):
    """Every row of a ragged batch has the bits of its run alone."""
    counts = [0, 3, 40, 9, 300]
    k, n = 640, 160
    ids, offsets, rows, pos, q, s = _product_case(counts, k, seed=9)
    w = Experts(tq, len(counts), n, k, fmt, seed=33)
    y = bits(tq.moe_gemv(w.dev, cuda(q), cuda(s), tq.MoePlan(cuda(offsets), cuda(rows), cuda(pos)), gather=True))
    for r in list(range(0, 20)) + [60, 200, int(offsets[-1]) - 1]:
        e = int(np.searchsorted(offsets, r, side="right") - 1)
        one = tq.moe_plan(cuda(np.array([[e]], np.int32)), len(counts))
        alone = bits(tq.moe_gemv(w.dev, cuda(q[rows[r]][None]), cuda(s[rows[r]][None]), one))
        assert np.array_equal(alone[0], y[r]), r


def test_a_bad_plan_is_clamped(tq):
    """Offsets and rows out of range reach no memory outside the arrays."""
    import torch
    w = Experts(tq, 3, 64, 256, 0, seed=1)
    q, s = act(4, 256)
    y = torch.zeros((8 + 4, 64), device="cuda")                       # 4 rows behind the 8 slots stay 0
    offsets = np.array([-5, 4, 2, 1 << 30], np.int32)
    rows = np.array([0, 9, -7, 3, 1 << 30, 1, 2, 3], np.int32)
    plan = tq.MoePlan(cuda(offsets), cuda(rows), cuda(np.zeros((4, 2), np.int32)))
    tq.moe_gemv(w.dev, cuda(q), cuda(s), plan, gather=True, y=y[:8])
    torch.cuda.synchronize()
    assert (y[8:] == 0).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("rows", [8, 512])
def test_offsets_that_do_not_ascend_have_no_rows(tq, rows):
    """Overlapping shares would add up to more rows than there are: nothing is written."""
    import torch
    w = Experts(tq, 3, 64, 256, 0, seed=1)
    q, s = act(rows, 256)
    y = torch.full((rows, 64), -1.0, device="cuda")
    order = cuda(np.arange(rows, dtype=np.int32).reshape(rows, 1))
    plan = tq.MoePlan(cuda(np.array([0, rows, 1, rows], np.int32)), order, order)
    tq.moe_gemv(w.dev, cuda(q), cuda(s), plan, y=y)
    torch.cuda.synchronize()
    assert (y == -1.0).all()


@pytest.mark.parametrize("m,topk,experts", [(9000, 8, 33), (70000, 2, 1000), (300000, 5, 8)])
def test_plan_of_many_chunks(tq, m, topk, experts):
    """The sort's counts are summed over many chunks of slots; every slot has one place."""
    rng = np.random.default_rng(m)
    ids = rng.integers(-1, experts, (m, topk)).astype(np.int32)
    plan = tq.moe_plan(cuda(ids), experts)
    order = np.argsort(np.where(ids.ravel() < 0, experts, ids.ravel()), kind="stable")
    total = int((ids >= 0).sum())
    pos = np.full(m * topk, -1, np.int32)
    pos[order[:total]] = np.arange(total, dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[ids >= 0], minlength=experts))])
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.pos.cpu().numpy().ravel(), pos)
    assert np.array_equal(plan.rows.cpu().numpy().ravel()[:total], order[:total] // topk)
    assert (plan.rows.cpu().numpy().ravel()[total:] == -1).all()


# ----------------------------------------------------------------------------
# sum over experts, and the layer
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("m,topk,n", [(1, 1, 4), (3, 8, 128), (65, 5, 516)])
def test_combine(tq, m, topk, n, bf16):
    import torch
    rng = np.random.default_rng(m)
    slots = m * topk
    y = rng.standard_normal((slots, n)).astype(np.float32)
    pos = rng.permutation(slots).astype(np.int32).reshape(m, topk)
    pos[rng.random((m, topk)) < 0.2] = -1
    if slots > 1:
        pos[0, 0] = slots + 5                                         # out of range: left out
    w = rng.random((m, topk)).astype(np.float32)
    plan = tq.MoePlan(None, cuda(np.zeros(slots, np.int32)), cuda(pos))
    out = tq.moe_combine(cuda(y), plan, cuda(w), dtype=torch.bfloat16 if bf16 else None)
    ok = ((pos >= 0) & (pos < slots))[..., None]
    t = np.where(ok, w[..., None].astype(np.float64) * y[np.clip(pos, 0, slots - 1)], 0)
    ref, mag = t.sum(1), np.abs(t).sum(1)
    tol = 1.01 * topk * U * mag + (2.0 ** -8 * 1.01 * np.abs(ref) if bf16 else 0) + 1e-40
    assert (np.abs(out.float().cpu().numpy() - ref) <= tol).all()


def _layer(tq, experts, hidden, inter, fmt):
    return tuple(Experts(tq, experts, n, k, fmt, seed=sd).dev
                 for n, k, sd in ((inter, hidden, 1), (inter, hidden, 301), (hidden, inter, 601)))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("m,experts,topk,hidden,inter", [(1, 8, 2, 256, 128), (7, 5, 3, 384, 256), (150, 4, 2, 256, 384)])
def test_ffn_is_its_parts_and_replays_in_a_graph(tq, m, experts, topk, hidden, inter, fmt):
    import torch
    gate, up, down = _layer(tq, experts, hidden, inter, fmt)
    ws = tq.moe_workspace(m, topk, experts, hidden, inter)
    stream = torch.cuda.Stream()
    outs = {}
    x = [torch.empty((m, hidden), device="cuda"), torch.empty((m, experts), device="cuda")]

    def step():
        res, q, s = tq.add_rmsnorm_rotq(x[0])
        ids, w = tq.moe_route(x[1], topk)
        return tq.moe_ffn(gate, up, down, q, s, ids, w, dtype=torch.bfloat16, workspace=ws)

    def parts():
        res, q, s = tq.add_rmsnorm_rotq(x[0])
        ids, w = tq.moe_route(x[1], topk)
        plan = tq.moe_plan(ids, experts)
        h = tq.moe_gateup(gate, up, q, s, plan)
        hq, hs = tq.rotate_quant(h)
        return tq.moe_combine(tq.moe_gemv(down, hq, hs, plan), plan, w, dtype=torch.bfloat16)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x[0].copy_(torch.randn(x[0].shape, generator=g, device="cuda"))
        x[1].copy_(torch.randn(x[1].shape, generator=g, device="cuda"))

    for seed in (1, 2):
        fill(seed)
        outs[seed] = parts()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):                               # a stream of its own
            got = step()
        stream.synchronize()
        assert torch.equal(got, outs[seed]) and torch.isfinite(got).all() and got.abs().max() > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in (2, 1, 2):                                            # other routings through one graph
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, outs[seed]), seed
    assert tq.read_error_word(ws[:4]) == 0


def test_layer_without_experts_is_zero(tq):
    import torch
    gate, up, down = _layer(tq, 3, 256, 128, 0)
    q, s = act(2, 256)
    ids = cuda(np.full((2, 2), -1, np.int32))
    y = tq.moe_ffn(gate, up, down, cuda(q), cuda(s), ids, torch.zeros((2, 2), device="cuda"))
    assert (y == 0).all()
