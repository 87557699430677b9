"""fp64 oracle of what surrounds a stage's block: linear maps with an epilogue,
layer norm, embedding.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).  Plain numpy in float64,
written from the definitions:

* linear: D = X W or X W^T; D + b + R, GeLU(D + b) + R or D GeLU'(H) + R;
* layer norm: y = gamma (x - mean) / sqrt(var + eps) + beta over each row, its
  gradient to the input from the full Jacobian's two projections, its gradients
  to gamma and beta as sums over rows;
* embedding: scaled rows of a table by id, the tokens in the order (id, token),
  the table's gradient one token after the other.
"""

from __future__ import annotations

import numpy as np

from . import block as ob


def linear(X, W, transposed=False, form="store", bias=None, R=None, H=None, tanh=False):
    """(out, D + bias)."""
    D = X @ (W.T if transposed else W)
    if bias is not None:
        D = D + bias
    act = "gelu_tanh" if tanh else "gelu_erf"
    out = D
    if form == "gelu":
        out = ob.gelu(D, act)
    elif form == "grad":
        out = D * ob.gelu_prime(H, act)
    return (out if R is None else out + R), D


def norm_stats(X, eps):
    mean = X.mean(axis=1)
    return mean, 1.0 / np.sqrt(((X - mean[:, None]) ** 2).mean(axis=1) + eps)


def norm_forward(X, gamma, beta, eps):
    mean, rstd = norm_stats(X, eps)
    y = (X - mean[:, None]) * rstd[:, None] * gamma
    return (y if beta is None else y + beta), mean, rstd


def norm_backward_input(dY, X, gamma, mean, rstd, dR=None):
    xh = (X - mean[:, None]) * rstd[:, None]
    u = dY * gamma
    dx = rstd[:, None] * (u - u.mean(axis=1, keepdims=True) - xh * (u * xh).mean(axis=1, keepdims=True))
    return dx if dR is None else dx + dR


def norm_backward_weight(dY, X, mean, rstd):
    xh = (X - mean[:, None]) * rstd[:, None]
    return (dY * xh).sum(axis=0), dY.sum(axis=0)


def embedding(ids, E, scale):
    Y = np.zeros((len(ids), E.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < len(E):
            Y[t] = scale * E[v]
    return Y


def embedding_order(ids, vocab):
    """(order, sorted_id)."""
    key = [int(v) if 0 <= v < vocab else vocab for v in ids]
    order = sorted(range(len(key)), key=lambda t: (key[t], t))
    return np.array(order, np.int64), np.array([key[t] if key[t] < vocab else -1 for t in order], np.int64)


def embedding_backward(ids, vocab, dY, scale):
    dE = np.zeros((vocab, dY.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < vocab:
            dE[v] += dY[t]
    return scale * dE
