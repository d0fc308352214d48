"""4-bit products at the ends of what one tile of rows holds: 176 rows where scales and minima are in the matrix
instructions (the columns up to the minima's own), 192 where they are folded, and one row more."""
import pytest

from test_q4_gpu import Matrix, _check, _x, no_wait_has_run_out, tq  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def product(w, x):
    """(x W^T, a bound of the kernel's error in fp32), both float64, for either form of the minima.

    Scales in the matrix instructions: 128 values are 16 of these, and the minima two more; each may drop bits below
    2^-23 of the largest of its 16 terms and of what it adds to (so 2 steps of 2^-23), over magnitudes that the two
    parts of a scale make up to 33/32 of their sum: 2 * 18 * 33/32 < 38 steps.  Behind it, as for the fold: 128
    additions of the sums of x, two roundings per group, the rounded 8 s - b, 2^-24 of its product with the sums, and the
    parts of a split along k; all relative to the sum of the magnitudes."""
    s = w.scales.double().repeat_interleave(w.group, 1)
    c, x = w.codes.double(), x.double()
    b = 8 * s if w.mins is None else w.mins.double().repeat_interleave(w.group, 1)
    size = x.abs() @ (s * (c - 8).abs()).T + x.abs() @ (8 * s - b).abs().T
    return x @ (s * c - b).T, (38 * 2.0 ** -23 + (128 + 2 * w.k // w.group + 27) * 2.0 ** -24) * size


@pytest.mark.parametrize("mins", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(131, 640), (1000, 2048), (20_001, 256)])
def test_rows_at_the_ends_of_a_tile(tq, n, k, group, mins):  # noqa: F811
    import torch
    w, up = Matrix(tq, n, k, group, mins, 11), Matrix(tq, n, k, group, mins, 12)
    for m in (160, 161, 175, 176, 177, 191, 192, 193, 352, 353, 384, 385):
        x = _x(m, k, m)
        want, tol = product(w, x)
        _check(tq.q4_gemv(w.dev, x), want, tol)
        need = tq.q4_workspace_bytes(m, k, group)                    # a workspace that is exactly as large, and what is behind it
        buf = torch.full((need + 512,), 90, dtype=torch.uint8, device="cuda")
        buf = buf[-buf.data_ptr() % 256:]
        _check(tq.q4_gemv(w.dev, x, workspace=buf[:need]), want, tol)
        assert (buf[need:] == 90).all()
        u, tu = product(up, x)
        s = want * want.sigmoid()
        tol = 1.1 * tol * (u.abs() + tu) + s.abs() * tu + 2.0 ** -20 * (s * u).abs()    # as test_q4_gpu.test_gateup
        _check(tq.q4_gateup(w.dev, up.dev, x), s * u, tol + 2.0 ** -8 * ((s * u).abs() + tol) + 1e-37)
