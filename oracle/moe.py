"""fp64 oracle of the mixture-of-experts operators and the 8-bit products.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).  Plain numpy in float64,
written from the definitions:

* router: the k largest logits of a row (ties to the lowest index, -inf never,
  NaN after every number), gates = softmax over all logits or over the chosen
  ones; rows ordered by (expert, token); the gates' gradient by the softmax's
  Jacobian;
* dispatch / combine: Xp[row(t, j)] = X[t], Y[t] = sum_j g[t, j] Yp[row(t, j)]
  and their gradients;
* experts: ``oracle.block`` on each expert's rows;
* 8 bits: e4m3 values (4 exponent bits with bias 7, 3 mantissa bits, subnormal
  step 2^-9, largest 448) with the least power-of-two scale that keeps a block
  of 128 within 448.
"""

from __future__ import annotations

import numpy as np

from . import block as ob


# --------------------------------------------------------------------------
# router
# --------------------------------------------------------------------------
def route(logits, k: int, renorm: bool):
    """Returns (gates, expert, offsets, row_of, token_of)."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    gates = np.zeros((T, k))
    expert = np.full((T, k), -1, np.int64)
    for t in range(T):
        # numbers by descending value, then NaNs; ties by index; -inf left out
        order = sorted((i for i in range(E) if not z[t, i] == -np.inf),
                       key=lambda i: (1, 0.0, i) if np.isnan(z[t, i]) else (0, -z[t, i], i))[:k]
        expert[t, :len(order)] = order
        if not order:
            continue
        if np.isnan(z[t]).any() or np.isposinf(z[t]).any():
            gates[t, :len(order)] = np.nan
            continue
        over = z[t, order] if renorm else z[t]
        top = z[t, order[0]]
        gates[t, :len(order)] = np.exp(z[t, order] - top) / np.exp(over - top).sum()
    counts = np.array([(expert == e).sum() for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    row_of = np.full((T, k), -1, np.int64)
    token_of = np.full(T * k, -1, np.int64)
    free = offsets[:-1].copy()
    for t in range(T):
        for j in range(k):
            e = expert[t, j]
            if e >= 0:
                row_of[t, j] = free[e]
                token_of[free[e]] = t
                free[e] += 1
    return gates, expert, offsets, row_of, token_of


def route_backward(logits, expert, dgates, renorm: bool):
    """d(sum of gates * dgates) / d logits by the softmax's full Jacobian."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    dz = np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(expert.shape[1]) if expert[t, j] >= 0]
        if not on:
            continue
        idx = [expert[t, j] for j in on] if renorm else list(range(E))
        e = np.exp(z[t, idx] - z[t, idx].max())
        p = e / e.sum()
        d = np.zeros(len(idx))
        for j in on:
            d[idx.index(expert[t, j])] = dgates[t, j]
        dz[t, idx] = (np.diag(p) - np.outer(p, p)) @ d
    return dz


# --------------------------------------------------------------------------
# rows
# --------------------------------------------------------------------------
def combine(Yp, row_of, gates=None):
    T, k = row_of.shape
    Y = np.zeros((T, Yp.shape[1]))
    for t in range(T):
        for j in range(k):
            if row_of[t, j] >= 0:
                Y[t] += (1.0 if gates is None else gates[t, j]) * Yp[row_of[t, j]]
    return Y


def combine_backward(dY, Yp, row_of, gates):
    """Returns (dYp, dgates); rows that nobody owns stay NaN."""
    dYp = np.full(Yp.shape, np.nan)
    dg = np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j in range(row_of.shape[1]):
            r = row_of[t, j]
            if r >= 0:
                dYp[r] = gates[t, j] * dY[t]
                dg[t, j] = dY[t] @ Yp[r]
    return dYp, dg


# --------------------------------------------------------------------------
# 8 bits
# --------------------------------------------------------------------------
def block_scale(amax):
    """Least power of two s >= 2^-126 with amax / s <= 448; 1 for 0, NaN for inf and NaN."""
    if not np.isfinite(amax):
        return np.nan
    if amax == 0:
        return 1.0
    s = 2.0 ** -126
    while amax / s > 448.0:
        s *= 2.0
    return s


def e4m3(x):
    """x rounded to e4m3, ties to even (|x| <= 448 expected), as float64."""
    x = np.asarray(x, np.float64)
    _, ex = np.frexp(np.abs(x))
    step = np.exp2(np.maximum(ex - 1, -6) - 3.0)  # 3 mantissa bits; subnormal step 2^-9
    return np.rint(x / step) * step


def quantize_rows(X):
    """Returns (values q as float64, scales)."""
    R, K = X.shape
    nb = -(-K // 128)
    q, S = np.zeros((R, K)), np.zeros((R, nb))
    for r in range(R):
        for b in range(nb):
            blk = X[r, b * 128:(b + 1) * 128]
            S[r, b] = block_scale(np.max(np.abs(blk)))
            q[r, b * 128:(b + 1) * 128] = e4m3(blk / S[r, b])
    return q, S


def quantize_weight(W):
    """W [rows, cols] in 128 x 128 blocks: (values q, scales)."""
    R, K = W.shape
    rb, cb = -(-R // 128), -(-K // 128)
    q, S = np.zeros((R, K)), np.zeros((rb, cb))
    for i in range(rb):
        for j in range(cb):
            at = (slice(i * 128, (i + 1) * 128), slice(j * 128, (j + 1) * 128))
            S[i, j] = block_scale(np.max(np.abs(W[at])))
            q[at] = e4m3(W[at] / S[i, j])
    return q, S


def spread_scales(S, rows, cols, row_block):
    """Scales of blocks (row_block x 128) spread over [rows, cols]."""
    return np.repeat(np.repeat(S, row_block, axis=0), 128, axis=1)[:rows, :cols]


# --------------------------------------------------------------------------
# experts
# --------------------------------------------------------------------------
def spans(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def by_expert(offsets, A, W, bias=None):
    """Rows of expert e times W[e] (+ bias[e]); rows past offsets[-1] are NaN.
    Also the sums of absolute products, for element-wise error bounds."""
    out = np.full((A.shape[0], W.shape[2]), np.nan)
    mag = np.zeros_like(out)
    for e, a, b in spans(offsets):
        if b > a:
            out[a:b] = A[a:b] @ W[e]
            mag[a:b] = np.abs(A[a:b]) @ np.abs(W[e])
            if bias is not None:
                out[a:b] += bias[e]
                mag[a:b] += np.abs(bias[e])
    return out, mag


gelu, gelu_prime = ob.gelu, ob.gelu_prime


# --------------------------------------------------------------------------
# a whole layer
# --------------------------------------------------------------------------
def layer_forward(X, logits, k, renorm, W1, W2, act="gelu_erf"):
    """Router, dispatch, experts and combine: (out, everything B and W need)."""
    gates, expert, offsets, row_of, token_of = route(logits, k, renorm)
    Xp = X[token_of[:int(offsets[-1])]]
    H, _ = by_expert(offsets, Xp, W1)
    A = gelu(H, act)
    Y, _ = by_expert(offsets, A, W2)
    return combine(Y, row_of, gates), dict(gates=gates, expert=expert, offsets=offsets, row_of=row_of, X=Xp, H=H, A=A,
                                           Y=Y)


def layer_backward(dout, logits, renorm, W1, W2, s, act="gelu_erf"):
    """Gradients of sum(out * dout): (dX, dlogits, dW1, dW2)."""
    dY, dg = combine_backward(dout, s["Y"], s["row_of"], s["gates"])
    dA, _ = by_expert(s["offsets"], dY, W2.transpose(0, 2, 1))
    dH = dA * gelu_prime(s["H"], act)
    dXp, _ = by_expert(s["offsets"], dH, W1.transpose(0, 2, 1))
    dW1, dW2 = np.zeros_like(W1), np.zeros_like(W2)
    for e, a, b in spans(s["offsets"]):
        dW1[e] = s["X"][a:b].T @ dH[a:b]
        dW2[e] = s["A"][a:b].T @ dY[a:b]
    return combine(dXp, s["row_of"]), route_backward(logits, s["expert"], dg, renorm), dW1, dW2
