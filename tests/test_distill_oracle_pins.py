"""Pins of the float64 distillation oracle: hand-worked values, the closed
form with a full list, non-negativity, and its gradient against differences
of its loss."""

import numpy as np
import pytest

from oracle.distill_oracle import distill_row


def test_hand_worked_row():
    # student uniform over 4; teacher list: columns 2 and 0 with odds 3 : 1
    r = distill_row([0.0] * 4, [np.log(3.0), 0.0], [2, 0])
    assert r["loss"] == pytest.approx(0.75 * np.log(3.0) + 0.25 * np.log(1.0))
    assert r["grad"] == pytest.approx([0.25 - 0.25, 0.25, 0.25 - 0.75, 0.25])
    # the same list as half of the teacher's mass; the other half in one bucket
    r = distill_row([0.0] * 4, [np.log(3.0), 0.0], [2, 0], teacher_lse=np.log(8.0))
    p = [3 / 8, 1 / 8]
    assert r["loss"] == pytest.approx(sum(a * np.log(a / 0.25) for a in p) + 0.5 * np.log(0.5 / 0.5), abs=1e-15)
    assert r["grad"] == pytest.approx([0.25 - 1 / 8, 0.0, 0.25 - 3 / 8, 0.0])


def test_full_list_is_the_divergence():
    g = np.random.default_rng(3)
    s, t, tau = g.normal(size=9), g.normal(size=9), 1.7
    p = np.exp(t / tau) / np.exp(t / tau).sum()
    q = np.exp(s / tau) / np.exp(s / tau).sum()
    for lse in (None, np.log(np.exp(t / tau).sum())):
        r = distill_row(s, t, np.arange(9), tau, lse, 0.3)
        assert r["loss"] == pytest.approx(0.3 * tau ** 2 * np.sum(p * np.log(p / q)))
        assert r["grad"] == pytest.approx(0.3 * tau * (q - p))


def test_equal_models_and_empty_rows():
    g = np.random.default_rng(4)
    s = g.normal(size=50)
    top = np.argsort(-s)[:7]
    r = distill_row(s, s[top], top, 2.0, np.log(np.exp(s / 2.0).sum()))
    assert abs(r["loss"]) < 1e-14 and np.abs(r["grad"]).max() < 1e-15
    assert distill_row(s, s[top], np.full(7, -1))["loss"] == 0.0
    assert not distill_row(s, s[top], top, weight=0.0)["grad"].any()
    assert distill_row(s, [-np.inf, -np.inf], [3, 4])["loss"] == 0.0
    assert np.isnan(distill_row(s, [1.0, 2.0], [3, 50])["loss"])


@pytest.mark.parametrize("full_mass", [False, True])
@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_gradient_is_the_loss_difference(tau, full_mass):
    g = np.random.default_rng(5)
    V = 12
    s, t = g.normal(size=V), 2 * g.normal(size=V)
    idx = np.array([3, 7, -1, 0, 7])  # an empty slot, and a column listed twice
    lse = np.log(np.exp(t / tau).sum()) + 0.7 if full_mass else None
    r = distill_row(s, t[idx], idx, tau, lse, 0.8)
    # with a renormalised list the masses of its columns add up; a list that
    # repeats a column still has p summing to 1
    h = 1e-5
    for j in range(V):
        e = np.zeros(V)
        e[j] = h
        d = (distill_row(s + e, t[idx], idx, tau, lse, 0.8)["loss"] -
             distill_row(s - e, t[idx], idx, tau, lse, 0.8)["loss"]) / (2 * h)
        assert d == pytest.approx(r["grad"][j], abs=1e-9)
