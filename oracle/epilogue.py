"""The linear layer's epilogue and its backward in float64.

``z = C + bias``, ``y = act(z) + residual``; ``dz = dy act'(z)``,
``dbias = sum over rows``.  The derivative of relu at 0 is 0; gelu is the tanh
form.
"""

import numpy as np

GELU_C = np.sqrt(2.0 / np.pi)
GELU_A = 0.044715


def _sigmoid(x):
    # no overflow on either side
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * _sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + np.tanh(GELU_C * (z + GELU_A * z ** 3)))
    assert name == "none"
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = _sigmoid(z)
        return s + z * s * _sigmoid(-z)
    if name == "gelu":
        t = np.tanh(GELU_C * (z + GELU_A * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * z ** 2)
    assert name == "none"
    return np.ones_like(z)


def forward(C, bias, name, residual):
    """(y, z) of the product's sums C [M][N]."""
    z = C if bias is None else C + bias
    y = act(z, name)
    return (y if residual is None else y + residual), z


def backward(dy, z, name):
    """(dz, dbias)."""
    dz = dy * act_grad(z, name)
    return dz, dz.sum(axis=0)
