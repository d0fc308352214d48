"""Sampling against the rule of include/tq_sample.h in 64 bits: the drawn tokens have to be equal."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def tq():
    from ternary_weight_dp4a_gb300 import build
    from ternary_weight_dp4a_gb300 import tq as m
    build.build()
    return m


def rule(logits, biggest, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row (float64 values of the stored logits) -> (id, probability)."""
    l = np.where(np.isnan(logits), -INF, np.minimum(logits, biggest))
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -INF]
    if len(order) == 0:
        return -1, 0.0
    if not t >= 2.0 ** -99:
        return int(order[0]), 1.0
    if 0 < top_k < len(order):
        order = order[:top_k]
    w = np.exp((l[order] - l[order[0]]) / t) if t < INF else np.ones(len(order))
    if min_p > 0:
        stay = max(1, int((w >= min(min_p, 1.0)).sum()))
        order, w = order[:stay], w[:stay]
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        stay = max(1, int((before < max(top_p, 0.0) * w.sum()).sum()))
        order, w = order[:stay], w[:stay]
    by_index = np.argsort(order)
    order, w = order[by_index], w[by_index]
    u = min(max(u, 0.0), 1.0) if u == u else 0.0
    c = np.cumsum(w)
    at = min(int((c <= u * c[-1]).sum()), len(w) - 1)
    return int(order[at]), float(w[at] / c[-1])


def check(tq, logits, u, **settings):
    """Compare all rows; `settings` are arrays [m] or None."""
    import torch
    f32 = lambda v, d=torch.float32: None if v is None else torch.as_tensor(np.asarray(v), dtype=d, device="cuda")  # noqa: E731
    s = {k: f32(v, torch.int32 if k == "top_k" else torch.float32) for k, v in settings.items()}
    uniform = f32(u)
    ids, probs = tq.sample(logits, uniform, **s)
    host = logits.double().cpu().numpy()
    biggest = torch.finfo(logits.dtype).max
    off = {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0}
    rows = {k: np.full(len(host), off[k]) if s.get(k) is None else s[k].double().cpu().numpy() for k in off}
    for r in range(len(host)):
        want = rule(host[r], biggest, float(uniform[r]), rows["temperature"][r], int(rows["top_k"][r]), rows["top_p"][r], rows["min_p"][r])
        got = int(ids[r]), float(probs[r])
        assert got[0] == want[0], (r, got, want, {k: v[r] for k, v in rows.items()}, float(uniform[r]))
        # a weight's error of 2^-30, of its sum too, and half a step of fp32
        assert abs(got[1] - want[1]) <= want[1] * (2.0 ** -24 + 2.0 ** -29) + 2.0 ** -40, (r, got, want)
    return ids, probs


def _logits(m, vocab, spread, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (spread * torch.randn((m, vocab), generator=g, device="cuda")).to(getattr(torch, dtype))


VOCABS = [1, 2, 31, 32, 33, 511, 513, 4097, 8192, 8193, 32003, 131072, 300_001]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_all_settings(tq, vocab, dtype):
    rng = np.random.default_rng(vocab)
    m = 24 if vocab < 100_000 else 8
    logits = _logits(m, vocab, 3.0, dtype, vocab)
    u = rng.random(m, dtype=np.float32)
    t = rng.uniform(0.3, 1.5, m).astype(np.float32)
    k = rng.integers(0, 200, m)
    p = rng.uniform(0.05, 1.05, m).astype(np.float32)
    f = rng.uniform(0, 0.2, m).astype(np.float32)
    check(tq, logits, u)
    check(tq, logits, u, temperature=t)
    check(tq, logits, u, temperature=t, top_k=k)
    check(tq, logits, u, temperature=t, top_p=p)
    check(tq, logits, u, temperature=t, min_p=f)
    check(tq, logits, u, temperature=t, top_k=k, top_p=p, min_p=f)
    check(tq, logits, u, temperature=t * (k % 3 > 0), top_k=k, top_p=p * (k % 2 > 0), min_p=f * (k % 4 > 0))


@pytest.mark.parametrize("vocab", [7, 513, 40_000])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.3, 30.0, 1e4])
def test_flat_and_steep_rows(tq, vocab, spread):
    rng = np.random.default_rng(1)
    m = 16
    u = rng.random(m, dtype=np.float32)
    for dtype in ("float32", "bfloat16"):
        logits = _logits(m, vocab, spread, dtype, 5)
        for k, p in ((0, 1.0), (0, 0.7), (50, 1.0), (vocab - 1, 0.5)):
            check(tq, logits, u, top_k=np.full(m, k), top_p=np.full(m, p))


def test_borders_of_equal_weights_are_met_exactly(tq):
    """Equal logits: sums are whole multiples, and a target that equals one decides as the rule says."""
    import torch
    m, vocab = 8, 1000
    logits = torch.zeros((m, vocab), device="cuda")
    u = np.arange(m) / 8.0                              # u * 1000 = 125 r: the index 125 r itself
    ids, probs = check(tq, logits, u)
    assert ids.tolist() == [125 * r for r in range(m)] and (probs == 0.001).all()
    ids, _ = check(tq, logits, np.full(m, 0.99999994), top_p=np.arange(1, m + 1) / 8)
    assert ids.tolist() == [125 * r - 1 for r in range(1, m + 1)]
    ids, _ = check(tq, logits, np.full(m, 0.99999994), top_k=np.arange(1, m + 1))
    assert ids.tolist() == list(range(m))
    logits[:, 400:] = 5.0                               # ties at the cut, behind other indices
    ids, _ = check(tq, logits, np.full(m, 0.99999994), top_k=np.arange(1, m + 1))
    assert ids.tolist() == [400 + r for r in range(m)]


def test_masked_entries(tq):
    import torch
    low = torch.finfo(torch.float32).min
    for dtype in ("float32", "bfloat16"):
        logits = _logits(9, 700, 2.0, dtype, 3)
        low = torch.finfo(logits.dtype).min
        logits[0] = -INF                                # nothing is left
        logits[1] = float("nan")
        logits[2] = -INF
        logits[2, 613] = low                            # one candidate, of the lowest value
        logits[3] = low                                 # all of them
        logits[4, ::2] = low
        logits[5, ::2] = -INF
        logits[5, 1::4] = float("nan")
        logits[6, 17] = INF
        logits[7, [17, 400]] = INF                      # two largest
        logits[8, 5] = torch.finfo(logits.dtype).max    # counts as much as +infinity
        logits[8, 3] = INF
        u = np.full(9, 0.7, np.float32)
        ids, probs = check(tq, logits, u)
        assert ids[0] == -1 and ids[1] == -1 and probs[0] == 0 and probs[1] == 0 and ids[2] == 613 and ids[6] == 17
        assert ids[7] == 400 and ids[8] == 5 and probs[8] == 0.5
        for s in (dict(top_k=np.full(9, 3)), dict(top_p=np.full(9, 0.3)), dict(min_p=np.full(9, 0.5)), dict(temperature=np.zeros(9)),
                  dict(temperature=np.full(9, INF), top_k=np.full(9, 600), top_p=np.full(9, 0.9), min_p=np.full(9, 1.0))):
            check(tq, logits, u, **s)


def test_settings_at_their_ends(tq):
    m, vocab = 12, 5000
    logits = _logits(m, vocab, 2.0, "float32", 3)
    u = np.random.default_rng(3).random(m, dtype=np.float32)
    nan = float("nan")
    t = [0.0, -1.0, nan, INF, 1e-30, 1e-29, 1e-3, 1e3, 1e30, 3e38, 1e-45, -0.0]
    check(tq, logits, u, temperature=t)
    check(tq, logits, u, temperature=t, top_k=np.arange(m), top_p=np.full(m, 0.5), min_p=np.full(m, 0.01))
    check(tq, logits, u, top_k=[-5, 0, 1, 2, vocab - 1, vocab, vocab + 1, 2**31 - 1, -2**31, 7, 7, 7])
    check(tq, logits, u, top_p=[-1.0, 0.0, 1e-45, 1e-20, 0.99999994, 1.0, 2.0, INF, -INF, nan, 0.5, 0.1])
    check(tq, logits, u, min_p=[-1.0, 0.0, 1e-45, 1e-38, 0.99999994, 1.0, 2.0, INF, -INF, nan, 0.5, 0.1])
    check(tq, logits, [0.0, -0.0, -1.0, nan, 1.0, 2.0, INF, -INF, 0.99999994, 1e-45, 1e-20, 0.5])
    check(tq, -logits.abs() * 1e38, u, temperature=np.full(m, 1e38))    # differences past the largest number


def test_zero_has_one_value(tq):
    import torch
    logits = torch.zeros((2, 64), device="cuda")
    logits[0, ::2] = -0.0
    logits[1, 1::2] = -0.0
    ids, _ = check(tq, logits, [0.3, 0.9], top_k=[5, 5])
    assert ids.tolist() == [1, 4]


def test_rows_do_not_depend_on_each_other(tq):
    import torch
    for vocab in (1000, 50_000):
        logits = _logits(40, vocab, 2.0, "bfloat16", 8)
        u = torch.rand((40,), device="cuda")
        t, p, k = torch.full((40,), 0.8, device="cuda"), torch.full((40,), 0.9, device="cuda"), torch.full((40,), 90, device="cuda", dtype=torch.int32)
        ids, probs = tq.sample(logits, u, t, k, p)
        for r in range(0, 40, 7):
            i, q = tq.sample(logits[r:r + 1], u[r:r + 1], t[:1], k[:1], p[:1])
            assert i.item() == ids[r].item() and q.item() == probs[r].item()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab", [4097, 9000, 20_000, 40_001, 70_001, 131_072])
def test_a_row_is_the_same_in_any_batch(tq, vocab, dtype):
    """Batches of other sizes give a row more or fewer CTAs, and its parts are kept or read again."""
    import torch
    rng = np.random.default_rng(vocab)
    most = 320
    logits = _logits(most, vocab, 2.5, dtype, 9)
    logits[::16] = logits[::16].round()                                     # many equal
    logits[3::16] = 1.0
    logits[5::16, ::2] = -INF
    logits[7::16, 1000:] = torch.finfo(logits.dtype).min
    logits[9::16, 100] = float("nan")
    logits[11::16] *= 1e-3
    on = lambda v, d=torch.float32: torch.as_tensor(v, dtype=d, device="cuda")  # noqa: E731
    u = on(rng.random(most, dtype=np.float32))
    t = on(rng.uniform(0.3, 1.5, most) * (rng.integers(0, 12, most) > 0))
    k = on(rng.integers(0, 700, most) * (rng.integers(0, 3, most) > 0), torch.int32)
    p = on(np.where(rng.integers(0, 3, most) > 0, rng.uniform(0.05, 1, most), 1.0))
    f = on(rng.uniform(0, 0.1, most) * (rng.integers(0, 2, most) > 0))
    for settings in ({}, {"temperature": t}, {"top_k": k}, {"top_p": p}, {"min_p": f}, {"temperature": t, "top_k": k, "top_p": p, "min_p": f}):
        few = [tq.sample(logits[i:i + 4], u[i:i + 4], **{n: v[i:i + 4] for n, v in settings.items()}) for i in range(0, most, 4)]
        ids, probs = (torch.cat(v) for v in zip(*few))
        for m in (20, 50, 76, 100, 160, most):
            got = tq.sample(logits[:m], u[:m], **{n: v[:m] for n, v in settings.items()})
            assert torch.equal(got[0], ids[:m]) and torch.equal(got[1], probs[:m]), (m, list(settings))


def test_shares_are_the_probabilities(tq):
    """Evenly spaced numbers draw every token as often as its probability says, within one."""
    import torch
    m, vocab = 4096, 50
    logits = _logits(1, vocab, 1.5, "float32", 2)
    u = (torch.arange(m, device="cuda") + 0.5) / m
    ids, probs = tq.sample(logits.expand(m, vocab).contiguous(), u, min_p=torch.full((m,), 0.02, device="cuda"))
    for token in ids.unique().tolist():
        at = ids == token
        assert abs(at.sum().item() - m * probs[at][0].item()) <= 1.0
    assert abs(sum(probs[ids == token][0].item() for token in ids.unique().tolist()) - 1) < 1e-5


def test_nothing_else_is_written_and_any_alignment_is_read(tq):
    import torch
    m, vocab = 5, 1237
    for dtype in (torch.float32, torch.bfloat16):
        base = _logits(1, m * vocab + 8, 2.0, str(dtype)[6:], 1)[0]
        for shift in range(4):
            logits = base[shift:shift + m * vocab].view(m, vocab)
            u = torch.rand((m,), device="cuda")
            buf, fbuf = torch.full((m + 8,), 77, dtype=torch.int32, device="cuda"), torch.full((m + 8,), 7.0, device="cuda")
            tq.sample(logits, u, ids=buf[3:3 + m], probs=fbuf[3:3 + m])
            ids, probs = check(tq, logits, u.cpu().numpy())
            assert torch.equal(buf[3:3 + m], ids) and torch.equal(fbuf[3:3 + m], probs)
            assert (buf[:3] == 77).all() and (buf[3 + m:] == 77).all() and (fbuf[:3] == 7).all() and (fbuf[3 + m:] == 7).all()


def test_streams_and_graphs(tq):
    import torch
    m, vocab = 6, 40_000
    rows = [_logits(m, vocab, 2.0, "float32", s) for s in range(3)]
    u = torch.rand((m,), device="cuda")
    p = torch.full((m,), 0.9, device="cuda")
    want = [tq.sample(l, u, top_p=p) for l in rows]
    logits = rows[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ids, probs = tq.sample(logits, u, top_p=p)
    for l, (i, q) in zip(rows, want):
        logits.copy_(l)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, i) and torch.equal(probs, q)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)
        logits.copy_(rows[1])
    i, q = tq.sample(logits, u, top_p=p, stream=other)
    other.synchronize()
    assert torch.equal(i, want[1][0]) and torch.equal(q, want[1][1])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_largest_vocabulary(tq, dtype):
    """One CTA has all of a row, in bins that pass 32 bits where the row is flat; few rows have eight."""
    import torch
    m, vocab = 160, 1 << 20
    logits = _logits(m, vocab, 1.0, dtype, 4)
    logits[::4] = 2.0
    logits[1::4] *= 4
    logits[2::4, 5:] = -2.0
    u = torch.rand((m,), device="cuda")
    for settings in ({}, {"top_p": 0.8}, {"top_k": 300}, {"top_k": 700_000, "top_p": 0.5, "min_p": 0.01}):
        on = {n: torch.full((m,), v, device="cuda", dtype=torch.int32 if n == "top_k" else torch.float32) for n, v in settings.items()}
        ids, probs = tq.sample(logits, u, **on)
        for r in (0, 4, 80):
            i, q = tq.sample(logits[r:r + 4], u[r:r + 4], **{n: v[r:r + 4] for n, v in on.items()})
            assert torch.equal(i, ids[r:r + 4]) and torch.equal(q, probs[r:r + 4])
        check(tq, logits[:4], u[:4].cpu().numpy(), **{n: v[:4].cpu().numpy() for n, v in on.items()})


def test_many_rows(tq):
    """More rows than CTAs that fit at once, and offsets past 32 bits."""
    import torch
    m, vocab = 20_000, 120_000
    logits = torch.zeros((m, vocab), dtype=torch.bfloat16, device="cuda")
    at = (torch.arange(m, device="cuda") * 7919) % vocab
    logits[torch.arange(m, device="cuda"), at] = 30.0
    ids, probs = tq.sample(logits, torch.full((m,), 0.5, device="cuda"), min_p=torch.full((m,), 0.1, device="cuda"))
    assert torch.equal(ids.long(), at) and (probs == 1).all()
