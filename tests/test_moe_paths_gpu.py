"""Products grouped by expert on each of the kernels that can run them: the same bits.

Which one runs depends on sizes alone (csrc/tq_moe_stream.cu, csrc/tq_moe_api.cu): few units
of 32 (gate/up: 16) weight rows take split_kernel, many take stream_kernel, experts with
many rows tile_kernel.  64 experts of 1000 outputs are on the stream kernel's side, one
token of them on the split kernel's, 49 rows for each of them on the tile kernel's.

Tolerances against 64 bits as in test_moe_gpu.py.  Where a gate is below -88.7 the
exponential overflows and SiLU is -0 instead of at most 89 e^-88.7 < 3e-37.
"""
import numpy as np
import pytest

from test_moe_gpu import U, act, bits, cuda, tq  # noqa: F401 (fixture)
from ternary_weight_dp4a_gb300 import synth

pytestmark = pytest.mark.gpu
B, E, N = 128, 64, 1000


class Weights:
    """E matrices [n][k] on the device, their scales at an address that is 2 mod 8 if `odd`."""

    def __init__(self, tq, n, k, fmt, seed, odd, scale=1.0):
        import torch
        mats = [synth.weight(n, k, fmt, seed + e) for e in range(E)]
        self.codes, self.n, self.k, self.fmt = np.stack([c for c, _ in mats]), n, k, fmt
        self.scales = (np.stack([s for _, s in mats]).astype(np.float64) * scale).astype(np.float16)
        dev = torch.empty(self.scales.size + 1, dtype=torch.float16, device="cuda")
        dev = dev[1:] if odd else dev[:-1]
        dev = dev.view(self.scales.shape)
        dev.copy_(cuda(self.scales))
        assert dev.data_ptr() % 8 == (2 if odd else 0)
        self.dev = tq.pack_experts(cuda(self.codes), fmt, dev)

    def terms(self, e, q, s):
        """Block terms d_b * scale_w * scale_a in 64 bits, [rows][n][nb] (d_b < 2^53: exact)."""
        c = self.codes[e].astype(np.float64)
        w = np.where(c == 2, -1, c) if self.fmt == 0 else 2 * c - 1
        nb = self.k // B
        d = np.matmul(q.astype(np.float64).reshape(len(q), nb, B).transpose(1, 0, 2),
                      w.reshape(self.n, nb, B).transpose(1, 2, 0)).transpose(1, 2, 0)
        return d * self.scales[e].astype(np.float64)[None] * s.astype(np.float64)[:, None, :]


def _counts(seed):
    """Rows of each expert: none, one, and around the chunks of eight; some beyond 32."""
    rng = np.random.default_rng(seed)
    c = rng.choice([0, 0, 1, 2, 3, 7, 8, 9, 16, 17, 25], E)
    c[[3, 17, 63]] = 33, 70, 5
    c[0] = 0
    assert 16 * E <= c.sum() + 16 * E and c.sum() < 2560                # the tile kernel is left out
    return c


def _sorted_plan(tq, counts):
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    order = cuda(np.arange(offsets[-1], dtype=np.int32))
    return offsets, tq.MoePlan(cuda(offsets), order, order)


def _on_tiles(tq, counts, q, s):
    """The same rows again and again until every expert that has some has 49; where they come from."""
    src, many = [], np.where(counts > 0, np.maximum(counts, 49), 0)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    many[np.argmax(counts)] += max(0, 49 * E - many.sum())               # 48 rows an expert and more on average
    for e in range(E):
        src.append(offsets[e] + np.arange(many[e]) % max(counts[e], 1))
    src = np.concatenate(src).astype(np.int64)
    _, plan = _sorted_plan(tq, many)
    assert len(src) > 48 * E
    return src, plan, cuda(q[src]), cuda(s[src])


def _alone(tq, counts, offsets, want, call):
    """Single rows: bits of call(expert, row) against want[row]."""
    for e in range(E):
        for r in {int(offsets[e]), int(offsets[e + 1]) - 1}:
            if counts[e] and e % 5 in (0, 2, 3):
                plan = tq.moe_plan(cuda(np.array([[e]], np.int32)), E)
                assert np.array_equal(call(r, plan)[0], want[r]), (e, r)


@pytest.mark.parametrize("k,odd", [(640, False), (1024, False), (1024, True), (1152, True)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_gemv_on_every_kernel(tq, fmt, k, odd):  # noqa: F811
    import torch
    counts = _counts(k + fmt)
    w = Weights(tq, N, k, fmt, 50, odd)
    offsets, plan = _sorted_plan(tq, counts)
    q, s = act(int(offsets[-1]), k, seed=k)
    q[::7, ::11] = -128
    y = torch.full((len(q), N), np.nan, device="cuda")
    tq.moe_gemv(w.dev, cuda(q), cuda(s), plan, y=y)                      # stream
    got = y.cpu().numpy().astype(np.float64)
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        t = w.terms(e, q[at], s[at])
        assert (np.abs(got[at] - t.sum(2)) <= 1.01 * (k // B + 1) * U * np.abs(t).sum(2) + 1e-44).all(), e
    want = bits(y)
    _alone(tq, counts, offsets, want,                                    # split
           lambda r, one: bits(tq.moe_gemv(w.dev, cuda(q[r][None]), cuda(s[r][None]), one)))
    src, many, qs, ss = _on_tiles(tq, counts, q, s)                      # tile
    assert np.array_equal(bits(tq.moe_gemv(w.dev, qs, ss, many)), want[src])


@pytest.mark.parametrize("k,odd", [(640, False), (1024, False), (1024, True), (1152, True)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_gateup_on_every_kernel(tq, fmt, k, odd):  # noqa: F811
    """Rows of ordinary size, and rows whose gates pass 64 on both sides, are zero, or are below
    2^-80 (where up is large enough for a product that bf16 holds)."""
    import torch
    counts = _counts(k + fmt + 1)
    g, u = Weights(tq, N, k, fmt, 150, odd, scale=2.0 ** -18), Weights(tq, N, k, fmt, 250, odd, scale=2.0 ** 20)
    offsets, plan = _sorted_plan(tq, counts)
    q, s = act(int(offsets[-1]), k, seed=k + 5)
    s[:] *= np.float32(2.0 ** 21)                                        # ordinary gates: a few units
    s[1::6] *= np.float32(2.0 ** 5)                                      # beyond 64
    s[2::6] *= np.float32(2.0 ** -84)                                    # below 2^-80
    q[3::6] = 0
    q[4::12, ::9] = -128
    h = torch.full((len(q), N), np.nan, device="cuda", dtype=torch.bfloat16)
    tq.moe_gateup(g.dev, u.dev, cuda(q), cuda(s), plan, gather=False, h=h)      # stream
    got = h.float().cpu().numpy().astype(np.float64)
    most, least, nb = 0.0, np.inf, k // B
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        tg, tu = (w.terms(e, q[at], s[at]) for w in (g, u))
        g64, u64 = tg.sum(2), tu.sum(2)
        dg, du = (1.01 * (nb + 1) * U * np.abs(t).sum(2) for t in (tg, tu))
        with np.errstate(over="ignore"):
            sil = g64 / (1 + np.exp(-g64))
        ref = sil * u64
        tol = (2.0 ** -8 + 8 * U) * np.abs(ref) + 1.01 * (1.1 * dg * np.abs(u64) + np.abs(sil) * du + 1.1 * dg * du) \
            + 3e-37 * (np.abs(u64) + du) + 1e-38
        assert (np.abs(got[at] - ref) <= tol).all(), e
        if g64.size:
            most = max(most, np.abs(g64).max())
            least = min(least, np.abs(g64[g64 != 0]).min(initial=np.inf))
    assert most > 64 and least < 2.0 ** -80
    want = bits(h)
    _alone(tq, counts, offsets, want,                                    # split
           lambda r, one: bits(tq.moe_gateup(g.dev, u.dev, cuda(q[r][None]), cuda(s[r][None]), one)))
    src, many, qs, ss = _on_tiles(tq, counts, q, s)                      # tile
    assert np.array_equal(bits(tq.moe_gateup(g.dev, u.dev, qs, ss, many, gather=False)), want[src])


def _bad_plan(slots, experts, rows, seed):
    """Ascending offsets and rows, both with entries out of range, and what they are clamped to."""
    rng = np.random.default_rng(seed)
    inner = np.sort(rng.integers(0, slots, experts - 1))
    offsets = np.concatenate([[-5], inner, [1 << 30]]).astype(np.int32)
    wild = rng.integers(-rows, 2 * rows, slots)
    wild[[0, -1]] = -(1 << 31), (1 << 31) - 1
    return offsets, np.clip(offsets, 0, slots).astype(np.int32), wild.astype(np.int32), np.clip(wild, 0, rows - 1).astype(np.int32)


# (experts, n, tokens, slots): split, stream, and tile (with the stream or split kernel beside it)
@pytest.mark.parametrize("experts,n,tokens,slots", [(3, 64, 4, 8), (64, 1000, 20, 100), (3, 64, 30, 512), (4, 520, 900, 2700)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_entries_out_of_range_are_clamped(tq, experts, n, tokens, slots, fmt):  # noqa: F811
    """Offsets and rows out of range stand for the nearest that are in range, and no row behind the
    last slot is written."""
    import torch
    k, guard = 384, 16
    gen = torch.Generator(device="cuda").manual_seed(7)
    w = []
    for _ in range(2):
        codes = torch.randint(0, 2, (experts, n, k), generator=gen, device="cuda", dtype=torch.uint8)
        scales = (0.01 + 0.04 * torch.rand((experts, n, k // B), generator=gen, device="cuda")).half()
        w.append(tq.pack_experts(codes, fmt, scales))
    q, s = (cuda(a) for a in act(tokens, k))
    offsets, offsets_ok, rows, rows_ok = _bad_plan(slots, experts, tokens, slots)
    bad, good = (tq.MoePlan(cuda(o), cuda(r), cuda(np.zeros(slots, np.int32))) for o, r in
                 ((offsets, rows), (offsets_ok, rows_ok)))
    y = torch.full((slots + guard, n), -1.0, device="cuda")
    tq.moe_gemv(w[0], q, s, bad, gather=True, y=y[:slots])
    assert np.array_equal(bits(y[:slots]), bits(tq.moe_gemv(w[0], q, s, good, gather=True))) and (y[slots:] == -1.0).all()
    h = torch.full((slots + guard, n), -1.0, device="cuda", dtype=torch.bfloat16)
    tq.moe_gateup(w[0], w[1], q, s, bad, h=h[:slots])
    assert np.array_equal(bits(h[:slots]), bits(tq.moe_gateup(w[0], w[1], q, s, good))) and (h[slots:] == -1.0).all()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("m", [5, 40, 700])
def test_layers_of_many_units(tq, m, fmt):  # noqa: F811
    """A whole FFN on the stream kernel (700 tokens: and the tile kernel) is its parts, and repeats."""
    import torch
    experts, topk, hidden, inter = E, 6, 1152, 640
    gen = torch.Generator(device="cuda").manual_seed(m)
    gate, up, down = (tq.pack_experts(torch.randint(0, 2, (experts, n, k), generator=gen, device="cuda", dtype=torch.uint8), fmt,
                                      (0.01 + 0.04 * torch.rand((experts, n, k // B), generator=gen, device="cuda")).half())
                      for n, k in ((inter, hidden), (inter, hidden), (hidden, inter)))
    ws = tq.moe_workspace(m, topk, experts, hidden, inter)
    logits = torch.randn((m, experts), generator=gen, device="cuda") + 2 * torch.randn((experts,), generator=gen, device="cuda")
    _, q, s = tq.add_rmsnorm_rotq(torch.randn((m, hidden), generator=gen, device="cuda"))
    ids, weights = tq.moe_route(logits, topk)
    y = tq.moe_ffn(gate, up, down, q, s, ids, weights, workspace=ws)
    plan = tq.moe_plan(ids, experts)
    hq, hs = tq.rotate_quant(tq.moe_gateup(gate, up, q, s, plan))
    parts = tq.moe_combine(tq.moe_gemv(down, hq, hs, plan), plan, weights)
    assert torch.equal(y, parts) and torch.isfinite(y).all() and y.abs().max() > 0
    for _ in range(3):
        ws[256:].random_(0, 256, generator=gen)                          # nothing of a call before is read
        assert torch.equal(tq.moe_ffn(gate, up, down, q, s, ids, weights, workspace=ws), y)
    assert tq.read_error_word(ws[:4]) == 0
