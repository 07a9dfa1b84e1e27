"""The gated product of a feed-forward block and its backward in float64.

``y = act(gate) * up``; ``dgate = dy up act'(gate)``, ``dup = dy act(gate)``.
Activations as the epilogue's.
"""

import numpy as np

from .epilogue import act as _act
from .epilogue import act_grad


def split(z):
    """(gate, up): the halves of z's columns."""
    n = z.shape[1] // 2
    return z[:, :n], z[:, n:]


def forward(z, name):
    gate, up = split(z)
    return _act(gate, name) * up


def backward(dy, z, name):
    """dz = (dgate | dup)."""
    gate, up = split(z)
    return np.concatenate([dy * up * act_grad(gate, name), dy * _act(gate, name)], axis=1)
