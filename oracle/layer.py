"""A linear layer and the distillation loss over a teacher's top logits, each with its gradients.
TEST INFRASTRUCTURE.

[P1] section 三 and [P2] ZeRO Stage 3 name the passes a gathered layer is rebuilt for (forward, and
again for the backward) and print no arithmetic; the definitions are written out here in fp64, term
by term. Pinned in the CPU tests by torch's own layers, its kl_div and its automatic gradients, and by
central differences.
"""

from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_C, _A = math.sqrt(2.0 / math.pi), 0.044715
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(z):
    with np.errstate(over="ignore"):                     # exp past fp64: 0
        return 1.0 / (1.0 + np.exp(-z))


# The gates are written without 1 + erf and 1 + tanh, whose digits cancel for negative z:
# (1 + erf u)/2 = erfc(-u)/2 and (1 + tanh u)/2 = sigmoid(2u).


def act(z: np.ndarray, kind: str) -> np.ndarray:
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return z * _erfc(-z / math.sqrt(2.0)) / 2.0
    if kind == "gelu_tanh":
        return z * _sigmoid(2.0 * _C * (z + _A * z ** 3))
    if kind == "silu":
        return z * _sigmoid(z)
    return z


def act_slope(z: np.ndarray, kind: str) -> np.ndarray:
    """The slope; at an infinity its limit, 0 or 1."""
    z = np.clip(np.asarray(z, np.float64), -1e18, 1e18)  # both are reached long before; keeps a NaN
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return _erfc(-z / math.sqrt(2.0)) / 2.0 + z * np.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        u = 2.0 * _C * (z + _A * z ** 3)
        return _sigmoid(u) * (1.0 + z * _sigmoid(-u) * 2.0 * _C * (1.0 + 3.0 * _A * z * z))
    if kind == "silu":
        return _sigmoid(z) * (1.0 + z * _sigmoid(-z))
    return np.ones_like(z)


def linear_forward(x, w, bias=None, residual=None, kind="none"):
    """(y, z) before any rounding."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = act(z, kind)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, z


def linear_backward(dz, x, w):
    """(dx, dweight, dbias) of the pre-activation gradient dz."""
    dz = np.asarray(dz, np.float64)
    return dz @ np.asarray(w, np.float64), dz.T @ np.asarray(x, np.float64), dz.sum(0)


def distill(z, index, top, temperature, tail=None, weight=None):
    """(loss [rows], gradient [rows, vocab]) of the loss in the logits, row by row from the
    definition; the teacher entries of one index are added up first."""
    z, top = np.asarray(z, np.float64), np.asarray(top, np.float64)
    R, V = z.shape
    loss, grad = np.zeros(R), np.zeros((R, V))
    for r in range(R):
        w = 1.0 if weight is None else float(weight[r])
        rows = [(int(i), t / temperature) for i, t in zip(index[r], top[r]) if 0 <= i < V]
        rest = -math.inf if tail is None else float(tail[r])
        biggest = max([t for _, t in rows] + [rest])
        if w == 0.0 or biggest == -math.inf:
            continue
        if not z[r].max() > -math.inf or not z[r].max() < math.inf or np.isnan(z[r]).any():
            loss[r], grad[r] = math.nan, math.nan
            continue
        mass = [math.exp(t - biggest) for _, t in rows]
        mass_rest = math.exp(rest - biggest)
        total = math.fsum(mass + [mass_rest])
        y = z[r] / temperature
        e = np.exp(y - y.max())
        log_q = y - y.max() - math.log(e.sum())
        q = np.exp(log_q)
        p = np.zeros(V)
        kl = 0.0
        for (i, t), m in zip(rows, mass):
            if m > 0.0:
                p[i] += m / total
                kl += m / total * (t - biggest - math.log(total) - log_q[i])
        g = q - p
        if mass_rest > 0.0:
            outside = np.ones(V, bool)
            outside[[i for i, _ in rows]] = False
            q_rest = e[outside].sum() / e.sum()
            p_rest = mass_rest / total
            kl += p_rest * (math.log(p_rest) - (math.log(q_rest) if q_rest > 0 else -math.inf))
            if q_rest > 0:
                g[outside] -= p_rest * q[outside] / q_rest
        loss[r], grad[r] = w * kl, w / temperature * g
    return loss, grad
