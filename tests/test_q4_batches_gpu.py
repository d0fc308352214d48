"""Products whose k is split over a cluster, several batches of units one behind the other: every output against the
definition in 64 bits.

Calls of 9 to 16 rows split k from 5504 on (clusters of one up to 5632, of two up to 11264) and add up 8 units of 32 outputs
(gate/up: 16) at a time; calls of up to 8 rows split it from 11776 on, 32 units at a time.  152 clusters of one run at
once, 72 of two: the sizes below are three batches each, the last of which has one unit to six, or none in some clusters."""
import copy

import pytest

from test_q4_gpu import Matrix, _check, _x, no_wait_has_run_out, tq  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def product(w, x):
    """Matrix.product by blocks of weight rows: values and bounds of the kernel's error, float64 [m][n]."""
    import torch
    got = []
    for i in range(0, w.n, 16384):
        rows = copy.copy(w)
        rows.codes, rows.scales = w.codes[i:i + 16384], w.scales[i:i + 16384]
        rows.mins = None if w.mins is None else w.mins[i:i + 16384]
        got.append(rows.product(x))
    return torch.cat([y for y, _ in got], 1), torch.cat([tol for _, tol in got], 1)


@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k,rows", [(80_007, 5504, (9, 16)), (40_007, 6144, (9, 16)), (150_007, 11_776, (1, 8))])
def test_gemv(tq, n, k, rows, group, mins):  # noqa: F811
    import torch
    w = Matrix(tq, n, k, group, mins, n + k + group)
    x = _x(max(rows), k, group)
    want, tol = product(w, x)
    for m in rows:
        got = tq.q4_gemv(w.dev, x[:m])
        _check(got, want[:m], tol[:m])
        assert torch.equal(got, tq.q4_gemv(w.dev, x[:m]))
        _check(tq.q4_gemv(w.dev, x[:m], dtype=torch.bfloat16), want[:m], tol[:m] + 2.0 ** -8 * (want[:m].abs() + tol[:m]))
    if max(rows) <= 8:                                               # a row of a packed step has the bits that it has alone
        assert torch.equal(got[:1], tq.q4_gemv(w.dev, x[:1]))


@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k,rows", [(40_007, 5504, (9, 16)), (20_003, 6144, (9, 16)), (80_007, 11_776, (1, 8))])
def test_gateup(tq, n, k, rows, group, mins):  # noqa: F811
    import torch
    gate, up = Matrix(tq, n, k, group, mins, 1), Matrix(tq, n, k, group, mins, 2)
    x = _x(max(rows), k, group)
    g, tg = product(gate, x)
    u, tu = product(up, x)
    s = g * g.sigmoid()
    # |silu'| < 1.1; tq_silu and the product: a few roundings of fp32; half a step of bf16
    tol = 1.1 * tg * (u.abs() + tu) + s.abs() * tu + 2.0 ** -20 * (s * u).abs()
    tol += 2.0 ** -8 * ((s * u).abs() + tol) + 1e-37
    for m in rows:
        got = tq.q4_gateup(gate.dev, up.dev, x[:m])
        _check(got, (s * u)[:m], tol[:m])
        assert torch.equal(got, tq.q4_gateup(gate.dev, up.dev, x[:m]))
    if max(rows) <= 8:
        assert torch.equal(got[:1], tq.q4_gateup(gate.dev, up.dev, x[:1]))


def test_a_small_batch_repeats_itself(tq):  # noqa: F811
    """8 x 5120 x 17408, groups of 32 with minima, bf16: the same bits every time, alone or while other work runs, and as
    near to the definition as the bound says."""
    import torch
    w = Matrix(tq, 5120, 17408, 32, True, 3)
    x = _x(8, 17408, 3)
    want, tol = product(w, x)
    first = tq.q4_gemv(w.dev, x, dtype=torch.bfloat16)
    _check(first, want, tol + 2.0 ** -8 * (want.abs() + tol))
    exact = tq.q4_gemv(w.dev, x)
    assert torch.equal(exact.bfloat16(), first)                      # rounded once, at the end
    other = torch.cuda.Stream()
    for _ in range(50):
        tq.q4_gemv(w.dev, x, stream=other)
        assert torch.equal(tq.q4_gemv(w.dev, x, dtype=torch.bfloat16), first)
    other.synchronize()
