"""The losses' plain f64 forms: gradients against central differences, the
worked values of small cases, and the identities that the formulas imply."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import losses

STEP = 1e-6


def differences(f, x):
    """Central differences of f along each element of x (error about STEP^2)."""
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + STEP
        up = f()
        flat[i] = keep - STEP
        down = f()
        flat[i] = keep
        out[i] = (up - down) / (2 * STEP)
    return g


def close(a, b):
    assert np.all(np.abs(a - b) <= 1e-8 * (1 + np.abs(b).max())), np.abs(a - b).max()


@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_token_logp_gradient(temperature):
    rng = np.random.default_rng(1)
    x = rng.normal(0, 2, (4, 9))
    x[1, 3] = -np.inf
    target = np.array([2, 0, -1, 8])
    g, gh = rng.normal(size=4), rng.normal(size=4)
    _, lse, ent, _ = losses.token_logp(x, target, temperature)
    grad, _ = losses.token_logp_vjp(x, target, lse, g, ent, gh, temperature)

    def value():
        lp, _, h, _ = losses.token_logp(x, target, temperature)
        return (g * lp + gh * h)[target >= 0].sum()

    finite = np.isfinite(x)
    want = np.zeros_like(x)
    keep = x.copy()
    for i, k in zip(*np.nonzero(finite)):
        x[i, k] = keep[i, k] + STEP
        up = value()
        x[i, k] = keep[i, k] - STEP
        want[i, k] = (up - value()) / (2 * STEP)
        x[i, k] = keep[i, k]
    close(grad, want)
    assert grad[1, 3] == 0 and np.all(grad[2] == 0)


@pytest.mark.parametrize("squared,smooth,mean", [(False, 0.0, False), (False, 0.2, True), (True, 0.0, True)])
def test_pref_gradient(squared, smooth, mean):
    rng = np.random.default_rng(2)
    off = np.array([0, 3, 7, 7, 12])
    logp, ref = -rng.random(12), -rng.random(12)
    mask = rng.random(12) < 0.7
    f = lambda: losses.pref_loss(logp, ref, mask, off, 2, 0.3, smooth, squared, mean)[0]  # noqa: E731
    close(losses.pref_loss(logp, ref, mask, off, 2, 0.3, smooth, squared, mean)[3], differences(f, logp))


@pytest.mark.parametrize("seq_mean,token_adv", [(False, False), (True, True)])
def test_policy_gradient(seq_mean, token_adv):
    rng = np.random.default_rng(3)
    off = np.array([0, 5, 5, 14])
    logp = -rng.random(14)
    old = logp + rng.normal(0, 0.3, 14)
    ref = logp + rng.normal(0, 0.3, 14)
    mask = rng.random(14) < 0.8
    adv = rng.normal(size=14 if token_adv else 3)
    args = dict(kl_coef=0.2, seq_mean=seq_mean, token_adv=token_adv, hi=0.3)
    loss, counts, grad, _ = losses.policy_loss(logp, old, ref, adv, mask, off, 3, **args)
    close(grad, differences(lambda: losses.policy_loss(logp, old, ref, adv, mask, off, 3, **args)[0][0], logp))
    assert counts[0] == mask.sum()


def test_worked_values():
    # two tokens of probability 1/2 and 1/4 ... uniform logits over four entries
    lp, lse, ent, _ = losses.token_logp(np.zeros((1, 4)), np.array([1]))
    assert np.isclose(lp[0], -np.log(4)) and np.isclose(lse[0], np.log(4)) and np.isclose(ent[0], np.log(4))
    # equal answers: the margin is 0, the loss log 2, the slope -beta/2
    loss, each, reward, grad = losses.pref_loss(np.full(4, -1.0), np.full(4, -1.0), None, None, 1, 0.1)
    assert np.isclose(loss, np.log(2)) and np.allclose(grad, [-0.05, -0.05, 0.05, 0.05]) and np.all(reward == 0)
    # an unchanged policy: ratio 1, no clip, loss minus the mean advantage, KL 0
    lp = np.array([-1.0, -2.0])
    loss, counts, grad, _ = losses.policy_loss(lp, lp, lp, np.array([3.0]), None, None, 1, kl_coef=0.5)
    assert np.allclose(loss, [-3, -3, 0]) and np.array_equal(counts, [2, 0]) and np.allclose(grad, -1.5)


def test_clipped_tokens_have_no_policy_gradient():
    # ratios 1.5 and 0.5 with clip 0.2: held where moving further would gain
    lp = np.log([1.5, 0.5, 1.5, 0.5])
    loss, counts, grad, _ = losses.policy_loss(lp, np.zeros(4), None, np.array([1.0, 1.0, -1.0, -1.0]), None, None, 4,
                                               token_adv=True)
    assert np.array_equal(counts, [4, 2])
    assert np.allclose(grad * 4, [0, -0.5, 1.5, 0]) and np.isclose(loss[0] * 4, -1.2 - 0.5 + 1.5 + 0.8)


def test_rows_of_a_softmax_gradient_sum_to_nothing():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(3, 50))
    target = np.array([0, 7, 49])
    _, lse, ent, _ = losses.token_logp(x, target)
    grad, _ = losses.token_logp_vjp(x, target, lse, rng.normal(size=3), ent, rng.normal(size=3))
    assert np.abs(grad.sum(1)).max() < 1e-12
