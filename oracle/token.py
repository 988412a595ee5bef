"""Losses over the tokens of a batch, each with its gradient in the logits. TEST INFRASTRUCTURE.

Not on the pages (they name a layer's forward and backward and no loss); the definitions of the log
probability of a row's token, the clipped policy loss with a KL term and the preference loss of paired
answers are written out in fp64, row by row. Pinned in the CPU tests by torch's automatic gradients of the
same formulas and by central differences.
"""

from __future__ import annotations

import math

import numpy as np


def softmax(z, label, temperature=1.0):
    """(l [rows], dl/dz [rows, vocab]): 0 for a row without a token, NaN for one without a softmax."""
    z = np.asarray(z, np.float64)
    R, V = z.shape
    l, g = np.zeros(R), np.zeros((R, V))
    for r in range(R):
        y = int(label[r])
        if not 0 <= y < V:
            continue
        if np.isnan(z[r]).any() or not -math.inf < z[r].max() < math.inf:
            l[r], g[r] = math.nan, math.nan
            continue
        x = z[r] / temperature - z[r].max() / temperature
        e = np.exp(x)
        others = math.fsum(np.delete(e, y))
        total = others + e[y]
        l[r] = -math.log1p(others / e[y]) if e[y] > others else x[y] - math.log(total)
        g[r] = -e / total / temperature
        g[r, y] = others / total / temperature
    return l, g


def _expm1_less(d):
    """exp(d) - 1 - d by its series near 0."""
    if abs(d) > 0.5:
        return math.inf if d > 700 else math.expm1(d) - d
    term, total, k = d * d / 2, 0.0, 2
    while abs(term) > 1e-30 * abs(total) + 1e-300:
        total, k = total + term, k + 1
        term *= d / k
    return total


def policy(l, old, advantage, clip=(0.2, 0.2), ref=None, kl=0.0):
    """(loss, dloss/dl) of one token, without its weight."""
    if math.isnan(l):
        return math.nan, math.nan
    x = l - old
    ratio = math.exp(min(x, 700.0))
    low, high = 1.0 - clip[0], 1.0 + clip[1]
    loss, slope = 0.0, 0.0
    if advantage != 0.0:
        first = ratio * advantage
        second = min(max(ratio, low), high) * advantage
        loss = -min(first, second)
        slope = -first if first <= second else 0.0
    if ref is not None and kl != 0.0:
        d = ref - l
        loss += kl * _expm1_less(d)
        slope -= kl * math.expm1(min(d, 700.0))
    return loss, slope


def policy_rows(z, label, old, advantage, clip, ref, kl, weight, temperature):
    """(loss, l, dloss/dz) of every row."""
    l, g = softmax(z, label, temperature)
    loss = np.zeros(len(l))
    for r in range(len(l)):
        w = 1.0 if weight is None else float(weight[r])
        if w == 0.0 or not 0 <= int(label[r]) < np.shape(z)[1]:
            l[r], g[r] = 0.0, 0.0
            continue
        value, slope = policy(l[r], float(old[r]), float(advantage[r]), clip, None if ref is None else float(ref[r]), kl)
        loss[r] = w * value
        g[r] = 0.0 if slope == 0.0 else w * slope * g[r]
    return loss, l, g


def preference(l, on, start, beta, ref=None, weight=None, smoothing=0.0, margin=0.0, average=False):
    """(loss [pairs], sequences' l [2*pairs], dloss/dl [rows]) from the rows' l; on: whether a row has a token."""
    pairs = (len(start) - 1) // 2
    seq, n = np.zeros(2 * pairs), np.ones(2 * pairs)
    span = [slice(int(start[i]), max(int(start[i]), int(start[i + 1]))) for i in range(2 * pairs)]
    for i, s in enumerate(span):
        n[i] = max(1, int(np.sum(on[s]))) if average else 1
        seq[i] = math.fsum(np.asarray(l[s], np.float64)) / n[i]
    loss, slope = np.zeros(pairs), np.zeros(len(l))
    for p in range(pairs):
        w = 1.0 if weight is None else float(weight[p])
        if w == 0.0:
            continue
        gap = seq[2 * p] - seq[2 * p + 1] - (0.0 if ref is None else float(ref[2 * p]) - float(ref[2 * p + 1]))
        x = beta * gap - margin
        up = np.logaddexp(0.0, -x)
        loss[p] = w * ((1 - smoothing) * up + smoothing * np.logaddexp(0.0, x))
        rise = math.exp(-np.logaddexp(0.0, -x))
        fall = math.exp(-np.logaddexp(0.0, x))
        d = w * beta * (smoothing * rise - (1 - smoothing) * fall)
        slope[span[2 * p]] = d / n[2 * p]
        slope[span[2 * p + 1]] = -d / n[2 * p + 1]
    return loss, seq, np.where(on, slope, 0.0)
