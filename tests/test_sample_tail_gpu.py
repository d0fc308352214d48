"""Draws from a flat tail of tiny weights: what is lost by weights that are whole multiples of 2^-42 of the largest."""
import numpy as np
import pytest

from test_sample_gpu import tq  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -42
VOCAB = 1 << 20


@pytest.mark.parametrize("top_p", [None, 1 - 2.0 ** -24, 1 - 3 * 2.0 ** -24])
@pytest.mark.parametrize("peak", [0, VOCAB // 3, VOCAB - 1])
@pytest.mark.parametrize("units", [0.3, 0.49, 0.51, 1.0, 1.4, 1.6, 2.5, 40.3, 1000.7])
def test_one_peak_and_a_flat_tail(tq, units, peak, top_p):  # noqa: F811
    """The rule in real arithmetic and the kernel differ by 2^-43 (half a unit) and 2^-30 of it in each weight, so by E =
    vocab * 2^-43 + 2^-30 of the sum in each of the sums that decide: the kept sum, the draw's target and the sum up to an
    index.  A drawn index is right if the real sums around it reach within their errors of the real target; its probability
    if it lies within its weight's error and the sum's."""
    import torch
    m = 12
    l = np.float32(np.log(units * UNIT))
    logits = torch.full((m, VOCAB), float(l), device="cuda")
    logits[:, peak] = 0.0
    w = np.exp(float(l))                                             # of a tail entry, from the stored logit
    u = np.array([0.0, 0.5] + [1 - i * 2.0 ** -24 for i in range(1, m - 1)], np.float32)
    p = None if top_p is None else torch.full((m,), top_p, device="cuda")
    ids, probs = tq.sample(logits, torch.from_numpy(u).cuda(), top_p=p)
    total = 1 + (VOCAB - 1) * w
    error = VOCAB * UNIT / 2 + 2.0 ** -30 * total
    # the run that stays: the peak and the first tail entries by index until top_p of the sum is reached
    kept = VOCAB - 1 if top_p is None else min(VOCAB - 1, max(0, int(np.ceil((float(np.float32(top_p)) * total - 1) / w))))
    kept_sum = 1 + kept * w
    cut = 0.0 if top_p is None else 2 * error + w                    # the kept sum's own error, by where it ends
    for r in range(m):
        i, got = int(ids[r]), float(probs[r])
        mine = 1.0 if i == peak else w
        upto = (i + 1) * w if i < peak else 1 + i * w
        target = float(u[r]) * kept_sum
        slack = 3 * error + 2 * cut
        assert upto - mine <= target + slack and upto + slack >= target, (r, i, upto, target, slack)
        # w / sum: the weight's error, and the sum's relative to it; rounded to fp32
        assert abs(got - mine / kept_sum) <= UNIT / 2 + (2.0 ** -30 + 2.0 ** -24) * mine + (error + cut) * mine, (r, i, got, mine / kept_sum)
        if units < 0.5:                                              # nothing of the tail is left: never drawn
            assert i == peak and got == 1.0


@pytest.mark.parametrize("vocab", [5000, 131_072])
def test_weights_above_2_to_the_minus_13_have_the_relative_error(tq, vocab):  # noqa: F811
    """Half a unit is 2^-30 of 2^-13: above it, and with few candidates, only the relative error counts."""
    import torch
    m = 64
    rng = np.random.default_rng(vocab)
    logits = np.full((m, vocab), -np.inf, np.float32)
    for r in range(m):
        at = rng.choice(vocab, 40, replace=False)
        logits[r, at] = -rng.uniform(0, 9, 40)
        logits[r, at[0]] = 0
    u = rng.random(m, dtype=np.float32)
    ids, probs = tq.sample(torch.from_numpy(logits).cuda(), torch.from_numpy(u).cuda())
    w = np.exp(logits.astype(np.float64))
    c = np.cumsum(w, 1)
    for r in range(m):
        i = int(ids[r])
        target = float(u[r]) * c[r, -1]
        assert c[r, i] - w[r, i] <= target * (1 + 2.0 ** -27) and c[r, i] >= target * (1 - 2.0 ** -27)
        # both errors of its weight, and of the sum, and half a step of fp32
        assert abs(float(probs[r]) / (w[r, i] / c[r, -1]) - 1) <= 2.0 ** -24 + 4 * 2.0 ** -30
