"""Pins of oracle/stack.py: hand-worked values, closed forms and finite differences (CPU)."""

import numpy as np
import pytest

from oracle import stack as ref

H = 1e-6


def differences(fn, x):
    d = np.zeros_like(x)
    for i in range(x.size):
        up, down = x.copy(), x.copy()
        up.flat[i] += H
        down.flat[i] -= H
        d.flat[i] = (fn(up) - fn(down)) / (2 * H)
    return d


def test_norm_by_hand():
    # mean square of (3, 4, 0, 0, 0, 0, 0, 0) is 25 / 8, and eps makes it 4
    h = np.array([[3.0, 4, 0, 0, 0, 0, 0, 0]])
    assert np.allclose(ref.add_norm(h, np.full(8, 2.0), 0.875), h)


def test_log_softmax_by_hand():
    z = np.log(np.array([1.0, 2, 5, 0]).clip(1e-300)) + 7
    z[3] = -np.inf
    want = np.array([1, 2, 5]) / 8
    assert np.allclose(np.exp(ref.log_softmax(z)), [*want, 0])
    assert np.isclose(ref.entropy(ref.log_softmax(z)), -np.sum(want * np.log(want)))
    assert np.isclose(ref.entropy(ref.log_softmax(np.zeros(32))), np.log(32))
    assert (ref.log_softmax(np.full(3, -np.inf)) == -np.inf).all()


def test_top_by_hand():
    assert ref.top(np.array([1.0, 5, 5, -np.inf, 7, 5]), 4).tolist() == [4, 1, 2, 5]


def test_divergence_by_hand():
    logits = np.log(np.array([0.5, 0.25, 0.25]))
    # the teacher has both of its entries at 1/2: sum p log(p / q) = log(1/2 / 1/2) / 2 + log(1/2 / 1/4) / 2
    ids, values = np.array([0, 2, -1, 3]), np.array([1.0, 1.0, 9.0, 9.0])
    assert np.isclose(ref.distill(logits, 1.0, ids, values, False), np.log(2) / 2)
    # given as log probabilities that do not add up to 1, one of them twice
    values = np.log(np.array([0.25, 0.125, 1, 1]))
    ids = np.array([1, 1, -1, 3])
    assert np.isclose(ref.distill(logits, 1.0, ids, values, True), 0.25 * np.log(1) + 0.125 * np.log(0.5))
    assert ref.distill(logits, 1.0, np.array([-1]), np.array([1.0]), False) == 0


def test_no_divergence_from_itself():
    rng = np.random.default_rng(1)
    logits = rng.standard_normal(9)
    assert abs(ref.distill(logits, 0.7, np.arange(9), logits, False)) < 1e-15
    assert np.abs(ref.distill_backward(logits, 0.7, np.arange(9), logits, False, 1.0)).max() < 1e-15


def test_norm_gradient_is_the_differences():
    rng = np.random.default_rng(2)
    h, w, dy, dr = (rng.standard_normal(s) for s in ((3, 16), 16, (3, 16), (3, 16)))

    def loss(h_, w_):
        return np.sum(ref.add_norm(h_, w_, 1e-3) * dy) + np.sum(h_ * dr)

    dh, dw = ref.add_norm_backward(h, w, 1e-3, dy, dr)
    assert np.abs(dh - differences(lambda a: loss(a, w), h)).max() < 1e-8
    assert np.abs(dw - differences(lambda a: loss(h, a), w)).max() < 1e-8


@pytest.mark.parametrize("masked", [False, True])
def test_logprob_gradient_is_the_differences(masked):
    rng = np.random.default_rng(3)
    x, scale, g, f = rng.standard_normal(11) * 2, 1.3, 0.7, -0.4
    if masked:
        x[::3] = -np.inf

    def loss(z):
        logq = ref.log_softmax(z * scale)
        return g * logq[4] + f * ref.entropy(logq)

    with np.errstate(invalid="ignore"):
        want = differences(loss, x)
    want[x == -np.inf] = 0  # a masked logit stays masked
    assert np.abs(ref.logprobs_backward(x, scale, 4, g, f) - want).max() < 1e-8


@pytest.mark.parametrize("given", [False, True])
def test_divergence_gradient_is_the_differences(given):
    rng = np.random.default_rng(4)
    x, scale = rng.standard_normal(13), 0.8
    ids, values = np.array([3, 12, 3, -1, 0, 40]), rng.standard_normal(6) - 2
    want = differences(lambda z: 1.7 * ref.distill(z, scale, ids, values, given), x)
    assert np.abs(ref.distill_backward(x, scale, ids, values, given, 1.7) - want).max() < 1e-8
