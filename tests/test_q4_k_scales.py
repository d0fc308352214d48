"""What tq_q4.h says of Q4_K's scales: an fp16 number times a 6-bit one, rounded to fp16.  No GPU needed."""
import numpy as np


def test_a_product_of_17_bits_rounded_to_fp16_is_off_by_up_to_2_to_the_minus_11():
    d = np.arange(1, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float64)       # every positive fp16 number
    worst = 0.0
    for six in range(1, 64):
        exact = d * six
        exact = exact[exact < 65504]
        off = np.abs(exact.astype(np.float16).astype(np.float64) - exact)
        small = exact < 2.0 ** -14
        assert (off[small] <= 2.0 ** -25).all()
        worst = max(worst, float((off[~small] / exact[~small]).max()))
    assert 2.0 ** -11.1 < worst <= 2.0 ** -11
