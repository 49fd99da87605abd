"""Pins of the loss oracle (oracle/qrita_losses.py): probabilities that are
exact fractions, hand-worked clip and pair cases, gradients against central
differences, and planted mistakes that each fail a pin."""

import math

import numpy as np
import pytest

from oracle import dentropy, dlogp, policy_row, preference, row_softmax

LN2 = math.log(2.0)
# logits ln 1, ln 2, ln 4 (and ln 1): probabilities 1/8, 2/8, 4/8, 1/8
X = np.array([0.0, LN2, 2 * LN2, 0.0])
P = np.array([1, 2, 4, 1]) / 8.0


def test_probabilities_are_the_fractions():
    for t in range(4):
        r = row_softmax(X, None, t)
        assert np.allclose(r.p, P, atol=1e-15)
        assert r.logp == pytest.approx(math.log(P[t]), abs=1e-14)
        # H = -(1/8 ln 1/8) 2 - 1/4 ln 1/4 - 1/2 ln 1/2 = (6/8 + 4/8 + 4/8) ln 2
        assert r.entropy == pytest.approx(1.75 * LN2, abs=1e-14)
    # inv_t = 2 squares the weights: 1, 4, 16, 1
    assert np.allclose(row_softmax(X, None, 0, 2.0).p, np.array([1, 4, 16, 1]) / 22.0, atol=1e-15)
    # a kept set renormalises: {1, 3} has weights 2, 1
    r = row_softmax(X, [0, 1, 0, 1], 3)
    assert np.allclose(r.p, [0, 2 / 3, 0, 1 / 3], atol=1e-15) and r.logp == pytest.approx(-math.log(3.0))


def test_row_rules():
    assert row_softmax(X, None, -1).ignored and row_softmax(X, None, 4).ignored
    assert row_softmax(X, [1, 1, 0, 1], 2).logp == -np.inf  # token not kept
    r = row_softmax(X, [0, 0, 0, 0], 2)
    assert r.logp == -np.inf and r.entropy == 0 and not r.p.any() and not r.joins
    r = row_softmax([-np.inf] * 3, None, 0)
    assert r.logp == -np.inf and not r.joins
    r = row_softmax([1.0, -np.inf, 1.0], None, 1)
    assert r.logp == -np.inf and r.entropy == pytest.approx(LN2)
    assert np.isnan(row_softmax([1.0, np.nan], None, 0).logp)
    assert np.isnan(row_softmax([1.0, np.inf], None, 0).logp)
    # a NaN outside the kept set is never used
    assert row_softmax([0.0, np.nan, 0.0], [1, 0, 1], 0).logp == pytest.approx(-LN2)
    # rows of the type's lowest value are uniform
    assert np.allclose(row_softmax([np.finfo(np.float32).min] * 4, None, 1).p, 0.25)


@pytest.mark.parametrize("inv_t", [1.0, 0.6, 1.7])
def test_row_gradients_against_differences(inv_t):
    rng = np.random.default_rng(3)
    x = rng.standard_normal(9) * 2
    mask = np.ones(9, bool)
    mask[[2, 7]] = False
    for t in (0, 5):
        r = row_softmax(x, mask, t, inv_t)
        g, h = dlogp(r, t, inv_t), dentropy(r, inv_t)
        for j in range(9):
            e = np.zeros(9)
            e[j] = 1e-5
            up, dn = row_softmax(x + e, mask, t, inv_t), row_softmax(x - e, mask, t, inv_t)
            # central differences of step 1e-5 are off by about 1e-10
            assert g[j] == pytest.approx((up.logp - dn.logp) / 2e-5, abs=2e-9)
            assert h[j] == pytest.approx((up.entropy - dn.entropy) / 2e-5, abs=2e-9)


@pytest.mark.parametrize("adv,rho,loss,slope", [
    (2.0, 1.0, -2.0, -2.0),      # inside the clip: -A rho
    (2.0, 1.5, -2.4, 0.0),       # above it, A > 0: -A (1 + hi), no gradient
    (-2.0, 1.5, 3.0, 3.0),       # above it, A < 0: the unclipped term is the larger
    (-2.0, 0.5, 1.6, 0.0),       # below it, A < 0: -A (1 - lo), no gradient
    (2.0, 0.5, -1.0, -1.0),      # below it, A > 0
    (0.0, 1.5, 0.0, 0.0),
])
def test_clip_cases_by_hand(adv, rho, loss, slope):
    r = row_softmax(X, None, 1)
    got = policy_row(r, r.logp - math.log(rho), None, adv, 0.2, 0.2, 0.0, 0.0)
    assert got[0] == pytest.approx(loss, abs=1e-12) and got[2] == pytest.approx(slope, abs=1e-12) and got[1] == 0.0


def test_kl_and_entropy_by_hand():
    r = row_softmax(X, None, 1)  # logp = ln 1/4
    # ref = ln 1/2: e^q = 2, kl = 2 - ln 2 - 1, d kl / d logp = 1 - 2
    loss, kl, d, h = policy_row(r, None, math.log(0.5), 3.0, 0.2, 0.2, 0.5, 0.25)
    assert kl == pytest.approx(1 - LN2) and d == pytest.approx(-3.0 - 0.5) and h == -0.25
    assert loss == pytest.approx(-3.0 + 0.5 * (1 - LN2) - 0.25 * 1.75 * LN2)


def _policy_loss(x, mask, t, inv_t, old, ref, adv):
    return policy_row(row_softmax(x, mask, t, inv_t), old, ref, adv, 0.2, 0.3, 0.1, 0.05)[0]


def test_policy_gradient_against_differences():
    rng = np.random.default_rng(5)
    for trial in range(6):
        x = rng.standard_normal(7) * 2
        t = int(rng.integers(7))
        r = row_softmax(x, None, t, 1.3)
        old, ref, adv = r.logp + 0.3 * rng.standard_normal(), r.logp + 0.5 * rng.standard_normal(), float(rng.standard_normal())
        _, _, a, h = policy_row(r, old, ref, adv, 0.2, 0.3, 0.1, 0.05)
        g = a * dlogp(r, t, 1.3) + h * dentropy(r, 1.3)
        for j in range(7):
            e = np.zeros(7)
            e[j] = 1e-5
            num = (_policy_loss(x + e, None, t, 1.3, old, ref, adv) - _policy_loss(x - e, None, t, 1.3, old, ref, adv)) / 2e-5
            assert g[j] == pytest.approx(num, abs=1e-8)


def test_preference_by_hand():
    # logp of tokens 1, 2 and 0, 3: 1/4 * 1/2 against 1/8 * 1/8: ratio ln 8
    rows = [row_softmax(X, None, t) for t in (1, 2, 0, 3)]
    loss, pair, ratio, seq, coef = preference(rows, [0, 2, 4], None, None, 1.0)
    assert ratio[0] == pytest.approx(3 * LN2) and seq == pytest.approx([-3 * LN2, -6 * LN2])
    assert loss == pytest.approx(math.log1p(1 / 8)) and pair[0] == pytest.approx(loss)
    assert coef == pytest.approx([-1 / 9, -1 / 9, 1 / 9, 1 / 9])
    # means, a reference, a margin, smoothing: z = (ln 8 / 2 - 0.5) - 0.25
    loss, pair, ratio, seq, coef = preference(rows, [0, 2, 4], [0.5, 0.0], [2.0], 1.0, 0.1, 0.25, True)
    z = 1.5 * LN2 - 0.75
    assert ratio[0] == pytest.approx(1.5 * LN2 - 0.5)
    assert pair[0] == pytest.approx(0.9 * math.log1p(math.exp(-z)) + 0.1 * math.log1p(math.exp(z)))
    sig = 1 / (1 + math.exp(-z))
    assert coef[0] == pytest.approx(2 * (0.1 * sig - 0.9 * (1 - sig)) / 2) and loss == pytest.approx(2 * pair[0])
    # an ignored row and an empty sequence add nothing
    rows = [row_softmax(X, None, -1), row_softmax(X, None, 1)]
    loss, _, ratio, seq, coef = preference(rows, [0, 2, 2], None, None, 1.0)
    assert seq == pytest.approx([-2 * LN2, 0.0]) and coef[0] == 0 and coef[1] != 0


def test_preference_gradient_against_differences():
    rng = np.random.default_rng(9)
    starts = [0, 2, 3, 3, 6]
    x = rng.standard_normal((6, 5))
    t = rng.integers(0, 5, 6)
    ref = rng.standard_normal(4)

    def f(x):
        rows = [row_softmax(x[i], None, int(t[i])) for i in range(6)]
        return rows, preference(rows, starts, ref, [0.3, 0.9], 0.7, 0.2, 0.1, True)

    rows, out = f(x)
    for i in range(6):
        g = out[4][i] * dlogp(rows[i], int(t[i]), 1.0)
        for j in range(5):
            e = np.zeros((6, 5))
            e[i, j] = 1e-5
            assert g[j] == pytest.approx((f(x + e)[1][0] - f(x - e)[1][0]) / 2e-5, abs=1e-9)


def test_planted_mistakes_fail_a_pin():
    r = row_softmax(X, None, 1)
    g = dlogp(r, 1, 1.0)
    assert abs(g.sum()) < 1e-15 and abs((g - 2 * (np.arange(4) == 1)).sum()) > 1  # the token's own +1 once
    assert abs(dentropy(r, 1.0).sum()) < 1e-15  # a shift of all logits changes neither
    wrong = -r.p * np.log(r.p)  # the entropy left out of its own gradient
    assert abs(wrong.sum()) > 0.1
    # min for max in the clipped term gives the wrong sign of pessimism
    loss = policy_row(r, r.logp - math.log(1.5), None, 2.0, 0.2, 0.2, 0.0, 0.0)[0]
    assert loss != pytest.approx(min(-2.0 * 1.5, -2.0 * 1.2))
