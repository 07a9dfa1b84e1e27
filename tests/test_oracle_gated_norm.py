"""Pins of the norm's and the gated product's oracles: known values, torch's
float64 autograd and central differences."""

import numpy as np
import pytest
import torch

from oracle import gated, rmsnorm


def test_norm_known_values():
    h = np.array([[3.0, 4.0], [0.0, 0.0]])
    y, rstd = rmsnorm.forward(h, np.array([1.0, 2.0]), 0.5)
    assert np.allclose(rstd, [1 / np.sqrt(13.0), np.sqrt(2.0)], rtol=1e-15)
    assert np.allclose(y, [[3 / np.sqrt(13), 8 / np.sqrt(13)], [0, 0]], rtol=1e-15)


def test_norm_gradients():
    rng = np.random.default_rng(0)
    h, dy, g = rng.normal(size=(7, 40)), rng.normal(size=(7, 40)), rng.normal(size=40)
    _, rstd = rmsnorm.forward(h, g, 1e-3)
    dx, dg = rmsnorm.backward(dy, h, rstd, g)
    th, tg = torch.tensor(h, requires_grad=True), torch.tensor(g, requires_grad=True)
    y = th * torch.rsqrt((th * th).mean(dim=1, keepdim=True) + 1e-3) * tg
    y.backward(torch.tensor(dy))
    assert np.abs(dx - th.grad.numpy()).max() < 1e-13
    assert np.abs(dg - tg.grad.numpy()).max() < 1e-13
    u, e = rng.normal(size=h.shape), 1e-6
    f = lambda a: (rmsnorm.forward(a, g, 1e-3)[0] * dy).sum()
    assert abs((f(h + e * u) - f(h - e * u)) / (2 * e) - (dx * u).sum()) < 1e-7


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_gated_gradients(name):
    rng = np.random.default_rng(1)
    z, dy = 2 * rng.normal(size=(9, 24)), rng.normal(size=(9, 12))
    dz = gated.backward(dy, z, name)
    u, e = rng.normal(size=z.shape), 1e-6
    f = lambda a: (gated.forward(a, name) * dy).sum()
    assert abs((f(z + e * u) - f(z - e * u)) / (2 * e) - (dz * u).sum()) < 1e-7


def test_gated_known_values():
    z = np.array([[-1.0, 2.0, 5.0, 7.0]])
    assert gated.forward(z, "relu").tolist() == [[0.0, 14.0]]
    assert gated.forward(z, "none").tolist() == [[-5.0, 14.0]]
    assert gated.backward(np.ones((1, 2)), z, "relu").tolist() == [[0.0, 7.0, 0.0, 2.0]]
