"""The sum of x and 8 s - b as three bf16 each, and six of the nine products: restated in numpy.  No GPU needed."""
import numpy as np


def bf16(v):
    """fp32 rounded to bf16, to the nearest and ties to even."""
    u = v.view(np.uint32)
    return ((u + 0x7fff + (u >> 16 & 1)) & np.uint32(0xffff0000)).view(np.float32)


def parts(v):
    got, rest = [], v.copy()
    for _ in range(3):
        got.append(bf16(rest))
        rest = rest - got[-1]
    return got, rest


def test_three_parts_are_the_number():
    rng = np.random.default_rng(1)
    v = (rng.integers(1 << 23, 1 << 24, 1_000_000).astype(np.float32) * 2.0 ** -23).astype(np.float32)
    p, rest = parts(v)
    assert (rest == 0).all() and (sum(q.astype(np.float64) for q in p) == v).all()


def test_what_three_of_nine_products_come_to():
    """At most 2 * 2^-8 * 2^-17 + 2^-34 of the whole product: 2^-24, which numbers just above 1 + 2^-8 come close to."""
    rng = np.random.default_rng(2)
    some = rng.integers(1 << 23, 1 << 24, 200_000)
    close = (1 << 23) + (1 << 15) + np.arange(-600, 600)
    v = (np.concatenate([some, close]).astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float32)
    (_, v2, v3), _ = parts(v)
    worst = 0.0
    for other in (v, v[::-1].copy(), np.full_like(v, v[np.argmax(np.abs(v2.astype(np.float64) * v3))])):
        (_, w2, w3), _ = parts(other)
        left = v2.astype(np.float64) * w3 + v3.astype(np.float64) * w2 + v3.astype(np.float64) * w3
        worst = max(worst, float((np.abs(left) / (v.astype(np.float64) * other)).max()))
    assert worst <= 2.0 ** -24 + 2.0 ** -34
    assert worst > 2.0 ** -24.1
