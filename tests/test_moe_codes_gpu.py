"""Products grouped by expert over every int8 code, -128 included, exact on the tile kernel.

Weights of -1, 0, +1, scales of one and k = 512 make every product a whole number of at most
512 * 128 = 2^16: every fp32 step holds it exactly, so the comparison is for equality.
"""
import numpy as np
import pytest

from test_moe_gpu import cuda, tq  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
B = 128


def _codes(fmt, experts, n, k, rng):
    """Expert 0 random, expert 1 all +1, expert 2 all -1; the codes and the weights they stand for."""
    c = rng.integers(0, 3 if fmt == 0 else 2, (experts, n, k)).astype(np.uint8)
    c[1], c[2] = 1, 2 if fmt == 0 else 0
    v = c.astype(np.int64)
    return c, np.where(v == 2, -1, v) if fmt == 0 else 2 * v - 1


def _every_code(rows, k, rng):
    q = rng.integers(-128, 128, (rows, k)).astype(np.int8)
    q[0], q[1] = -128, 127
    q[2] = (np.arange(k) % 256 - 128).astype(np.int8)               # each code, twice
    q[3] = np.where(np.arange(k) % 2, 127, -128)
    q[4] = 0
    q[4, rng.integers(0, k)] = -128
    return q


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows", [2, 200])
def test_products_of_every_code(tq, fmt, rows):  # noqa: F811
    """200 rows of an expert run on the tile kernel, 2 on the others."""
    import torch
    n, k, experts = 130, 512, 3
    rng = np.random.default_rng(fmt + rows)
    codes, weights = _codes(fmt, experts, n, k, rng)
    w = tq.pack_experts(cuda(codes), fmt, torch.ones((experts, n, k // B), dtype=torch.float16, device="cuda"))
    q = _every_code(max(rows, 5), k, rng)[:rows] if rows >= 5 else _every_code(5, k, rng)[[0, 2]]
    q = np.concatenate([q] * experts)
    offsets = np.arange(experts + 1, dtype=np.int32) * rows
    order = cuda(np.arange(len(q), dtype=np.int32))
    plan = tq.MoePlan(cuda(offsets), order, order)
    y = tq.moe_gemv(w, cuda(q), torch.ones((len(q), k // B), device="cuda"), plan)
    ref = np.concatenate([q[rows * e:rows * (e + 1)].astype(np.int64) @ weights[e].T for e in range(experts)])
    bad = np.argwhere(y.cpu().numpy() != ref.astype(np.float32))
    assert len(bad) == 0, (len(bad), bad[:4].tolist())
