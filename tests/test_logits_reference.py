"""The 64-bit reference of the logits operators against itself: its gradients against central
differences of its values, and its values against closed forms (CPU only)."""
import math

import numpy as np
import pytest

import logits_reference as R


@pytest.mark.parametrize("cols", [1, 2, 7, 40])
@pytest.mark.parametrize("temperature", [1.0, 0.6, 2.5])
def test_logprob_gradient_is_the_difference(cols, temperature):
    rng = np.random.default_rng(cols)
    x = rng.normal(size=cols) * 2
    t, g, e = int(rng.integers(cols)), 0.7, -0.3

    def value(y):
        r = R.logprobs_row(y, t, temperature, 0)
        return g * r["logprob"] + e * r["entropy"]

    d, _ = R.logprobs_grad_row(R.logprobs_row(x, t, temperature, 0), x, t, temperature, g, e, "f32")
    step = 1e-5
    for j in range(cols):
        up, down = x.copy(), x.copy()
        up[j] += step
        down[j] -= step
        # the third derivative of a sum of such terms is at most about 30 / T^3
        assert abs((value(up) - value(down)) / (2 * step) - d[j]) < 30 / temperature ** 3 * step ** 2 + 1e-9


@pytest.mark.parametrize("k", [1, 3, 9])
def test_distillation_gradient_is_the_difference(k):
    rng = np.random.default_rng(k)
    cols, temperature, g = 23, 1.7, 1.3
    x = rng.normal(size=cols) * 2
    ids = rng.integers(0, cols, size=k)  # equal ids among them
    v = rng.normal(size=k) * 2
    if k > 3:
        ids[2] = -1
    d, _ = R.distill_grad_row(R.distill_row(x, ids, v, temperature), x, temperature, g, "f32")
    step = 1e-5
    for j in range(cols):
        up, down = x.copy(), x.copy()
        up[j] += step
        down[j] -= step
        diff = g * (R.distill_row(up, ids, v, temperature)["loss"] -
                    R.distill_row(down, ids, v, temperature)["loss"]) / (2 * step)
        assert abs(diff - d[j]) < 30 * step ** 2 + 1e-9


def test_closed_forms():
    r = R.logprobs_row(np.zeros(8), 3, 1.0, 3)
    assert abs(r["logprob"] + math.log(8)) < 1e-15 and abs(r["entropy"] - math.log(8)) < 1e-15
    assert [i for _, i in r["top"]] == [0, 1, 2]
    r = R.logprobs_row(np.array([-np.inf, 2.0, 2.0, -np.inf]), 1, 0.5, 3)
    assert abs(r["logprob"] + math.log(2)) < 1e-15 and r["top"][2] == (-math.inf, -1)
    # a teacher that equals the student on the whole vocabulary: no loss, no gradient
    x = np.array([0.3, -1.0, 2.0, 0.0])
    row = R.distill_row(x, np.arange(4), x, 1.3)
    d, _ = R.distill_grad_row(row, x, 1.3, 1.0, "f32")
    assert abs(row["loss"]) < 1e-15 and np.abs(d).max() < 1e-15
    # one entry: the negative log probability
    row = R.distill_row(x, np.array([2]), np.array([5.0]), 1.3)
    assert abs(row["loss"] + R.logprobs_row(x, 2, 1.3, 0)["logprob"]) < 1e-15
