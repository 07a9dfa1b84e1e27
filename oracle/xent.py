"""Softmax cross entropy of a head's logits and its gradients, in float64.

``l = x . w^T``; ``lse = log sum exp l``; ``loss = lse - l[target]``; a row
whose target is ``ignore_index`` or outside [0, V) has loss and lse 0 and takes
no part in the gradients, whatever its ``x`` holds.
"""

import numpy as np


def valid_rows(target, V, ignore_index=-100):
    target = np.asarray(target, dtype=np.int64)
    return (target != ignore_index) & (target >= 0) & (target < V)


def linear_xent(x, w, target, ignore_index=-100):
    """(loss, lse) [M] of float64 x [M][K], w [V][K]."""
    M, V = x.shape[0], w.shape[0]
    ok = valid_rows(target, V, ignore_index)
    loss, lse = np.zeros(M), np.zeros(M)
    for m in np.nonzero(ok)[0]:
        l = w @ x[m]
        top = l.max()
        lse[m] = top + np.log(np.exp(l - top).sum()) if np.isfinite(top) else top
        loss[m] = lse[m] - l[target[m]]
    return loss, lse


def softmax_minus_onehot(x, w, target, lse, ignore_index=-100):
    """G [valid rows][V] and the indices of those rows."""
    rows = np.nonzero(valid_rows(target, w.shape[0], ignore_index))[0]
    G = np.exp(x[rows] @ w.T - lse[rows][:, None])
    G[np.arange(rows.size), np.asarray(target)[rows]] -= 1.0
    return G, rows


def linear_xent_backward(x, w, target, lse, dloss, ignore_index=-100):
    """(dx [M][K], dw [V][K]) for gradients ``dloss`` [M] of the losses."""
    G, rows = softmax_minus_onehot(x, w, target, lse, ignore_index)
    G = G * dloss[rows][:, None]
    dx = np.zeros(x.shape)
    dx[rows] = G @ w
    return dx, G.T @ x[rows]
