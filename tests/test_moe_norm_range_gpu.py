"""The root of the norm at sums of squares near the end of binary32's range.

1/sqrt is to be the correctly rounded value but for about one row in 10^5.  The outputs are
bf16, so an error in its last bit is made visible by elements next to a border of bf16: per row
one element A carries the sum (the others' squares are below 2^-67 A^2 together), and for each
neighbour v of the true root w some elements t are such that bf16(t w) and bf16(t v) differ.
"""
import numpy as np
import pytest

from test_moe_gpu import bf16_round, cuda, tq  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def _rows(m, lo, hi, seed):
    """Residual rows [m][128] and the root of each, correctly rounded."""
    rng = np.random.default_rng(seed)
    a = np.sqrt(rng.uniform(lo, hi, m)).astype(np.float32)
    with np.errstate(over="ignore"):
        w = (1.0 / np.sqrt(a.astype(np.float64) ** 2 / 128)).astype(np.float32)
    # midpoints between neighbouring bf16 numbers, 2^-36 to 2^-35
    mid = (2.0 ** -36 * (1 + (2 * np.arange(127) + 1) / 256)).astype(np.float32)
    t = (mid[None, :] / w[:, None]).astype(np.float32)
    return np.concatenate([a[:, None], t], axis=1), w


def _shown(rows, w):
    """Whether a root one ulp above or below w would change a row's bf16 outputs."""
    x = bf16_round(rows * w[:, None])
    return [(bf16_round(rows * np.nextafter(w, np.float32(to))[:, None]) != x).any(1) for to in (0, 1)]


@pytest.mark.parametrize("lo,hi", [(1e4, 1e5), (1e30, 2e30), (1e34, 2e34), (1e36, 2e36), (9e36, 9.9e36), (1e37, 2e37)])
def test_root_is_correctly_rounded(tq, lo, hi):  # noqa: F811
    import torch
    m = 100_000
    rows, w = _rows(m, lo, hi, 3)
    below, above = _shown(rows[:2000], w[:2000])
    assert below.mean() > 0.99 and above.mean() > 0.99
    x = torch.empty((m, 128), dtype=torch.bfloat16, device="cuda")
    tq.add_rmsnorm_rotq(cuda(rows), eps=0.0, x_out=x)
    wrong = (x.float().cpu().numpy() != bf16_round(rows * w[:, None])).any(1)
    # one in 10^5 is expected at most: seven of 10^5 would be chance once in 10^4 runs
    assert wrong.sum() <= 6, int(wrong.sum())
