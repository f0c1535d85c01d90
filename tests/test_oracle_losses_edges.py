"""The plain f64 losses where a product of 0 and infinity decides."""
from __future__ import annotations

import numpy as np

from oracle import losses


def test_a_reference_that_is_only_watched():
    """kl_coef 0: the loss and its gradient are those without the reference, whatever it holds."""
    logp, old = np.array([-np.inf, -1.0, -2.0, -0.5]), np.full(4, -1.0)
    adv = np.array([0.5, -0.5])
    off = np.array([0, 2, 4])
    want = losses.policy_loss(logp, old, None, adv, None, off, 2)
    for ref in ([-2.0, -1.5, 800.0, 1e30], [-1.0, np.nan, np.inf, -np.inf]):
        got = losses.policy_loss(logp, old, np.array(ref), adv, None, off, 2)
        assert np.array_equal(got[0][:2], want[0][:2]) and np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])
        assert np.all(np.isfinite(got[2]))
    with_term = losses.policy_loss(logp[1:2], old[1:2], np.array([-0.5]), adv[:1], None, None, 1, kl_coef=0.25)
    assert np.isclose(with_term[2][0], -0.5 - 0.25 * np.expm1(0.5), rtol=1e-14)


def test_an_advantage_of_zero():
    """r A is 0 at A = 0 for every finite difference, also where r is beyond f64."""
    logp, old = np.full(5, -1.0), np.array([-800.0, -1e30, 1e30, -1.0, -1.5])
    for hi in (0.2, np.inf):
        loss, counts, grad, size = losses.policy_loss(logp, old, None, np.zeros(1), None, None, 1, hi=hi)
        assert np.all(loss == 0) and np.all(grad == 0) and np.all(size == 0) and counts.tolist() == [5, 0]
    loss, _, grad, _ = losses.policy_loss(logp, np.array([np.nan] * 5), None, np.zeros(1), None, None, 1)
    assert np.isnan(loss[0]) and np.all(np.isnan(grad))


def test_an_infinite_difference_to_the_reference():
    """exp(u) - u - 1 is infinite at both infinities of u."""
    for ref, logp in ((-1.0, -np.inf), (-np.inf, -1.0)):
        loss, _, _, _ = losses.policy_loss(np.array([logp]), np.array([-1.0]), np.array([ref]), np.ones(1), None, None, 1)
        assert loss[2] == np.inf and np.isfinite(loss[0])
