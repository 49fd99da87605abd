"""Pins of oracle/qrita_scores.py: exact probabilities, hand-worked orders,
differences against gradients, and agreement with the one-token oracle."""

import math

import numpy as np
import pytest

from oracle import cache_weights, kept_order, row_softmax, scores_grad_row, scores_row

LN = math.log


def test_exact_probabilities():
    # weights 4, 2, 1, 1, and one that is not kept
    x = [LN(2), LN(4), 0.0, 9.0, 0.0]
    logp, rank, H, ids, lp = scores_row(x, [1, 1, 1, 0, 1], [4, 1, 3, -1], top=6)
    assert np.allclose(logp, [LN(1 / 8), LN(1 / 2), -math.inf, 0.0])
    assert rank == 3  # behind 4, 2 and the equal logit of lower id
    assert H == pytest.approx(0.5 * LN(2) + 0.25 * LN(4) + 2 * 0.125 * LN(8))
    assert ids.tolist() == [1, 0, 2, 4, -1, -1]
    assert np.allclose(lp[:4], [LN(1 / 2), LN(1 / 4), LN(1 / 8), LN(1 / 8)]) and (lp[4:] == -math.inf).all()


def test_signed_zeros_and_unlikely_logits():
    x = [-0.0, 0.0, -math.inf, 1.0]
    _, rank, _, ids, _ = scores_row(x, None, [1], top=4)
    assert rank == 2 and ids.tolist() == [3, 0, 1, -1]
    assert scores_row(x, None, [2], top=1)[1] == -1
    assert scores_row(x, None, [7])[1] == -1


def test_empty_and_nan_rows():
    logp, rank, H, ids, lp = scores_row([1.0, 2.0], [0, 0], [1], top=1)
    assert logp[0] == -math.inf and rank == -1 and H == 0 and ids[0] == -1 and lp[0] == -math.inf
    logp, rank, H, ids, lp = scores_row([1.0, math.nan], None, [1, -1], top=1)
    assert math.isnan(logp[0]) and logp[1] == 0 and rank == -1 and math.isnan(H) and ids[0] == -1 and math.isnan(lp[0])
    assert scores_row([1.0, math.nan], [1, 0], [0])[0][0] == 0.0


def test_one_token_agrees_with_the_losses():
    rng = np.random.default_rng(1)
    x = rng.standard_normal(50) * 3
    mask = rng.random(50) < 0.6
    for t in range(50):
        want = row_softmax(x, mask, t, 0.7)
        got = scores_row(x, mask, [t], 0.7)
        assert got[0][0] == pytest.approx(want.logp) and got[2] == pytest.approx(want.entropy)


@pytest.mark.parametrize("inv_t", [1.0, 0.6])
def test_gradient_against_differences(inv_t):
    rng = np.random.default_rng(2)
    x = rng.standard_normal(12)
    mask = np.array([1] * 9 + [0] * 3)
    ids, g, h = [3, 7, 3, 10, -1, 0], np.array([0.4, -1.2, 0.9, 2.0, 5.0, 0.3]), -0.7

    def f(x):
        logp, _, H, _, _ = scores_row(x, mask, ids, inv_t)
        return sum(v * l for v, l in zip(g, logp) if l > -np.inf) + h * H

    got, _ = scores_grad_row(x, mask, ids, g, h, inv_t)
    for j in range(12):
        d = np.zeros(12)
        d[j] = 1e-5
        # central differences: off by d^2 / 6 of a third derivative below 10, and rounding of 1e-16 / 1e-5
        assert got[j] == pytest.approx((f(x + d) - f(x - d)) / 2e-5, abs=1e-8)


def test_cache_weights_by_hand():
    k = np.array([[LN(3)], [0.0], [LN(3)], [5.0]])
    q = np.ones((2, 1, 1))
    # positions 0, 1, 2; the first query sees two slots (3 : 1), the second all three (3 : 1 : 3)
    got = cache_weights(q, k, [0, 1, 2, 9], 3, 3, 1.0)
    assert np.allclose(got, [3 / 4 + 3 / 7, 1 / 4 + 1 / 7, 3 / 7])
    # a query of a position that no slot has reached sees nothing
    assert np.allclose(cache_weights(q, k, [0, 1, 2, 9], 1, 1, 1.0), [1.0])


def test_kept_order_by_hand():
    w = [0.5, math.nan, 0.5, 2.0, -0.0, 0.0, math.nan]
    at = [0, 1, 2, 3, 4, 5, 6]
    assert kept_order(w, at, 7, 7, 0, 0) == [3, 0, 2, 4, 5, 1, 6]
    assert kept_order(w, at, 7, 7, 2, 1) == [0, 1, 6, 3, 2, 4, 5]
    assert kept_order(w, at, 3, 7, 0, 0) == [0, 2, 1]
    # later tokens in early slots: the last two seen are positions 9 and 8
    assert kept_order([1, 2, 3], [9, 0, 8], 3, 10, 0, 2) == [2, 0, 1]


def test_planted_mistakes_are_seen():
    x = [1.0, 3.0, 3.0, 2.0]
    ids = scores_row(x, None, [2], top=3)
    assert ids[3].tolist() != [2, 1, 3] and ids[1] != 0  # ties to the higher id
    g, _ = scores_grad_row(x, None, [1, 1], [1.0, 1.0])
    once, _ = scores_grad_row(x, None, [1], [1.0])
    assert np.allclose(g, 2 * once) and not np.allclose(g, once)  # an id listed twice
