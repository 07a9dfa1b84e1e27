"""Pins of the epilogue oracle: known values, torch's float64 functions and
central differences."""

import numpy as np
import pytest
import torch

from oracle import epilogue


def test_against_torch():
    z = np.linspace(-12, 12, 4001)
    t = torch.from_numpy(z)
    for name, f in (("relu", torch.relu), ("silu", torch.nn.functional.silu),
                    ("gelu", lambda a: torch.nn.functional.gelu(a, approximate="tanh"))):
        assert np.abs(epilogue.act(z, name) - f(t).numpy()).max() < 1e-13


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_derivative_against_differences(name):
    z = np.linspace(-8.03, 8.05, 801)
    h = 1e-6
    d = (epilogue.act(z + h, name) - epilogue.act(z - h, name)) / (2 * h)
    assert np.abs(d - epilogue.act_grad(z, name)).max() < 1e-8


def test_known_values():
    assert epilogue.act(np.array([0.0]), "silu") == 0 and epilogue.act_grad(np.zeros(1), "relu") == 0
    assert abs(epilogue.act(np.array([1.0]), "silu")[0] - 1 / (1 + np.exp(-1.0))) < 1e-15
    assert epilogue.act_grad(np.zeros(1), "silu")[0] == 0.5
    assert epilogue.act_grad(np.zeros(1), "gelu")[0] == 0.5


def test_forward_order():
    """bias before the activation, the residual after it."""
    y, z = epilogue.forward(np.array([[-1.0]]), np.array([3.0]), "relu", np.array([[-5.0]]))
    assert z[0, 0] == 2 and y[0, 0] == -3
