"""Pins of oracle/updates.py: closed forms, the two forms of a step, and planted mistakes."""
import numpy as np
import pytest

from oracle import updates

RNG = np.random.default_rng(5)


def _poly(s, coefficients=updates.COEFFICIENTS, steps=5):
    for _ in range(steps):
        a, b, c = coefficients
        s = a * s + b * s ** 3 + c * s ** 5
    return s


@pytest.mark.parametrize("shape", [(7, 7), (12, 5), (5, 12), (1, 9), (9, 1), (1, 1)])
def test_singular_values_follow_the_scalar_polynomial(shape):
    u, s, vt = np.linalg.svd(RNG.normal(size=shape), full_matrices=False)
    got = updates.newton_schulz((u * s) @ vt)
    want = (u * _poly(s / np.linalg.norm(s))) @ vt
    assert np.abs(got - want).max() < 1e-12


def test_wide_is_the_transpose_of_tall():
    g = RNG.normal(size=(6, 11))
    assert np.abs(updates.newton_schulz(g) - updates.newton_schulz(g.T).T).max() < 1e-13


def test_scale_does_not_matter_and_zero_stays_zero():
    g = RNG.normal(size=(4, 6))
    assert np.abs(updates.newton_schulz(1e100 * g) - updates.newton_schulz(g)).max() < 1e-13
    assert not updates.newton_schulz(np.zeros((3, 4))).any()


def test_coefficients_for_each_step():
    s = np.array([0.3, 0.7, 0.2])
    rows = [(2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    want = s / np.linalg.norm(s)
    for r in rows:
        want = _poly(want, r, 1)
    assert np.abs(np.diag(updates.newton_schulz(np.diag(s), 2, rows)) - want).max() < 1e-13


def test_momentum_by_hand():
    g, b = np.array([[1.0, -2.0]]), np.array([[4.0, 8.0]])
    new, u = updates.momentum(g, b, 0.5)
    assert new.tolist() == [[3.0, 2.0]] and u.tolist() == [[2.5, -1.0]]
    assert updates.momentum(g, b, 0.5, nesterov=False)[1].tolist() == [[3.0, 2.0]]


@pytest.mark.parametrize("wrong", [(3.4445, 4.7750, 2.0315), (3.4445, -4.7750, -2.0315), (3.4445, -4.7750, 0.0)])
def test_planted_mistakes_fail_the_pin(wrong):
    u, s, vt = np.linalg.svd(RNG.normal(size=(8, 5)), full_matrices=False)
    got = updates.newton_schulz((u * s) @ vt, 1, wrong)
    assert np.abs(got - (u * _poly(s / np.linalg.norm(s), steps=1)) @ vt).max() > 1e-3
