"""The norms before and after a block with its gate and scales, and their gradients. TEST INFRASTRUCTURE.

The pages name a gathered layer's passes ([P1] section 三) and print no arithmetic; the definitions are written
out here in fp64. Pinned in the CPU tests by torch's layer_norm, its automatic gradients and central
differences.
"""

from __future__ import annotations

import numpy as np

KINDS = ("none", "rms", "layer")


def normalised(v, kind, eps):
    """(values in units of the row's deviation, mean, 1/deviation) of each row."""
    v = np.asarray(v, np.float64)
    zero, one = np.zeros((v.shape[0], 1)), np.ones((v.shape[0], 1))
    if kind == "none":
        return v, zero, one
    mean = v.mean(1, keepdims=True) if kind == "layer" else zero
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt(((v - mean) ** 2).mean(1, keepdims=True) + eps)
        return (v - mean) * rstd, mean, rstd


def affine(x, w, b):
    x = x if w is None else x * np.asarray(w, np.float64)
    return x if b is None else x + np.asarray(b, np.float64)


def spread(gate, rows, gate_rows):
    """The gate of each row."""
    return 1.0 if gate is None else np.asarray(gate, np.float64)[np.arange(rows) // gate_rows]


def forward_sum(x, branch, gate, gate_rows, post, post_w, post_b, eps, a, c):
    """y before its rounding."""
    if branch is None:
        return np.asarray(x, np.float64)
    value = affine(normalised(branch, post, eps)[0], post_w, post_b)
    return a * np.asarray(x, np.float64) + c * spread(gate, len(x), gate_rows) * value


def forward_next(y, pre, pre_w, pre_b, eps):
    """h of a y as it is stored."""
    return affine(normalised(y, pre, eps)[0], pre_w, pre_b)


def through(g, unit, rstd, kind):
    """The gradient in a norm's argument from the gradient g of its normalised values."""
    if kind == "none":
        return g
    rest = g.mean(1, keepdims=True) if kind == "layer" else 0.0
    return rstd * (g - rest - unit * (g * unit).mean(1, keepdims=True))


def backward(y, dy, dh, branch, gate, gate_rows, post, post_w, post_b, pre, pre_w, eps, a, c):
    """Every gradient, in a dict."""
    d = 0.0 if dy is None else np.asarray(dy, np.float64)
    out = {}
    if pre != "none":
        dh = np.asarray(dh, np.float64)
        xh, _, rstd = normalised(y, pre, eps)
        out["dpre_weight"], out["dpre_bias"] = (dh * xh).sum(0), dh.sum(0)
        d = d + through(affine(dh, pre_w, None), xh, rstd, pre)
    if branch is None:
        out["dx"] = d
        return out
    out["dx"] = a * d
    oh, _, rstd = normalised(branch, post, eps)
    rows = len(oh)
    each = c * d * affine(oh, post_w, post_b)
    if gate is not None:
        sums = np.zeros(np.shape(gate))
        np.add.at(sums, np.arange(rows) // gate_rows, each)
        out["dgate"] = sums
    e = c * spread(gate, rows, gate_rows) * d
    out["dpost_weight"], out["dpost_bias"] = (e * oh).sum(0), np.broadcast_to(e, oh.shape).sum(0)
    out["dbranch"] = through(affine(np.broadcast_to(e, oh.shape), post_w, None), oh, rstd, post)
    return out
