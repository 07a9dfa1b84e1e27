"""The root-mean-square norm and its backward in float64.

``y = h rstd g`` with ``rstd = 1 / sqrt(mean(h^2) + eps)`` over a row; with
``n = h rstd`` and ``u = g dy``, ``dx = rstd (u - n mean(u n))`` and
``dg = sum over the rows of dy n``.
"""

import numpy as np


def forward(h, g, eps):
    """(y, rstd)."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * g, rstd


def backward(dy, h, rstd, g):
    """(dx, dg)."""
    n = h * rstd[:, None]
    u = dy * g
    return rstd[:, None] * (u - n * (u * n).mean(axis=1, keepdims=True)), (dy * n).sum(axis=0)
