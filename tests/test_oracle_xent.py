"""Pins of the float64 cross-entropy oracle: a scalar brute force, closed
forms, and its gradients against central differences."""

import math

import numpy as np
import pytest

from oracle import xent


def _case(seed, M=5, V=7, K=4):
    r = np.random.default_rng(seed)
    return r.normal(size=(M, K)), r.normal(size=(V, K)), r.integers(0, V, size=M)


def test_scalar_brute_force():
    x, w, t = _case(0)
    loss, lse = xent.linear_xent(x, w, t)
    for m in range(5):
        l = [sum(x[m][k] * w[v][k] for k in range(4)) for v in range(7)]
        z = sum(math.exp(a) for a in l)
        assert abs(lse[m] - math.log(z)) < 1e-13
        assert abs(loss[m] + math.log(math.exp(l[t[m]]) / z)) < 1e-13


def test_equal_logits_give_log_v():
    w = np.ones((9, 3))
    loss, lse = xent.linear_xent(np.full((2, 3), 0.5), w, np.array([0, 8]))
    assert np.allclose(loss, math.log(9)) and np.allclose(lse, 1.5 + math.log(9))


@pytest.mark.parametrize("bad", [-100, -1, 7, 1 << 40])
def test_rows_without_a_loss(bad):
    x, w, t = _case(1)
    t[2] = bad
    x[2] = np.nan
    loss, lse = xent.linear_xent(x, w, t)
    assert loss[2] == 0 and lse[2] == 0 and np.all(np.isfinite(loss))
    dx, dw = xent.linear_xent_backward(x, w, t, lse, np.ones(5))
    assert np.all(dx[2] == 0) and np.all(np.isfinite(dw))


def test_gradients_against_differences():
    x, w, t = _case(2)
    t[1] = -100
    d = np.random.default_rng(3).normal(size=5)
    _, lse = xent.linear_xent(x, w, t)
    dx, dw = xent.linear_xent_backward(x, w, t, lse, d)
    h = 1e-6
    for a, g in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = (xent.linear_xent(x, w, t)[0] * d).sum()
            a[i] = keep - h
            down = (xent.linear_xent(x, w, t)[0] * d).sum()
            a[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-8


def test_planted_mistakes_show():
    """Leaving out the one-hot term or the row weights changes the result."""
    x, w, t = _case(4)
    _, lse = xent.linear_xent(x, w, t)
    d = np.array([1.0, 2.0, 0.5, 3.0, 1.0])
    dx, dw = xent.linear_xent_backward(x, w, t, lse, d)
    P = np.exp(x @ w.T - lse[:, None])
    assert np.abs(d[:, None] * (P @ w) - dx).max() > 0.1
    dx1, dw1 = xent.linear_xent_backward(x, w, t, lse, np.ones(5))
    assert np.abs(dw1 - dw).max() > 0.1 and np.abs(dx1 - dx).max() > 0.1
