"""4-bit products of large and small activations."""
import pytest

from test_q4_edges_gpu import product
from test_q4_gpu import Matrix, _check, _x, no_wait_has_run_out, tq  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bits", [117, -90])
def test_activations_up_to_the_stated_magnitude(tq, bits, group, mins):  # noqa: F811
    """All of one sign and of magnitudes up to 2^117: 8 * 128 * 2^117 is the largest that a group's sum gets, and what is added up
    here, at most 512 * 0.03 * 16 * 2^117 < 2^125, is in range as well.  (And small ones, far from the subnormal.)"""
    import torch
    w = Matrix(tq, 70, 512, group, mins, 21)
    for m in (1, 8, 9, 16, 17, 64, 100, 190):
        x = ((1 + _x(m, 512, m).float().abs().clamp(max=1)) * 2.0 ** (bits - 1)).bfloat16()
        assert float(x.float().abs().max()) == 2.0 ** bits
        for signed in (x, x * torch.where(_x(m, 512, 1) > 0, 1, -1).bfloat16()):
            want, tol = product(w, signed)
            got = tq.q4_gemv(w.dev, signed)
            assert got.isfinite().all()
            _check(got, want, tol)


@pytest.mark.parametrize("m", [1, 9, 40, 100])
@pytest.mark.parametrize("group,mins", [(32, False), (32, True), (128, True)])
def test_larger_ones_stay_in_their_rows(tq, group, mins, m):  # noqa: F811
    """Where a group's sum leaves fp32's range, its own row is infinite or NaN (or finite), and no other changes."""
    import torch
    w = Matrix(tq, 70, 512, group, mins, 22)
    x = _x(m, 512, m)
    clean = tq.q4_gemv(w.dev, x)
    row = m // 2
    x[row] = torch.finfo(torch.bfloat16).max
    got = tq.q4_gemv(w.dev, x)
    keep = torch.arange(m, device="cuda") != row
    assert torch.equal(got[keep], clean[keep])
