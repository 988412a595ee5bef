"""Adam's moments in 8 bits. TEST INFRASTRUCTURE.

The pages give the optimizer state 12 bytes a parameter ([P1] section 一); a form in 8 bits is not on
them, and the library's own definition is written out here, one fp32 operation at a time: blocks of 256
elements with one scale, the block's largest magnitude, and indices spaced as squares (127 of them with
a sign for m, 255 without for the root of v). Pinned in the CPU tests by a search over all indices and
by the spacing's own error bounds.
"""

from __future__ import annotations

import numpy as np

BLOCK = 256
F32 = np.float32


def _blocks(x: np.ndarray) -> np.ndarray:
    n = -(-x.size // BLOCK)
    out = np.zeros(n * BLOCK, x.dtype)
    out[:x.size] = x
    return out.reshape(n, BLOCK)


def encode(x: np.ndarray, top: int):
    """(codes, scale) of fp32 numbers: top 127 (int8, signed) or 255 (uint8, roots of the second moment)."""
    b = _blocks(np.ascontiguousarray(x, np.float32))
    mag = np.abs(b)
    scale = mag.max(1)                                   # a NaN in a block makes its scale NaN
    good = (scale >= F32(2.0 ** -126)) & (scale < np.inf)
    with np.errstate(all="ignore"):
        inv = F32(1.0) / np.where(good, scale, F32(1.0))
        t = (mag * inv[:, None]) * F32(top * top)
        q = np.ceil(np.sqrt(np.where(good[:, None], t, 0).astype(np.float64)) - 0.5)
    if top == 255:
        q = np.where((b > 0) & (q < 1), 1.0, q)
    q = np.where(good[:, None], q, 0.0)
    q = np.where(b < 0, -q, q) if top == 127 else q
    kept = np.where(good, scale, np.where(scale < F32(2.0 ** -126), F32(0.0), F32(np.nan)))
    return q.reshape(-1)[:x.size].astype(np.int8 if top == 127 else np.uint8), kept.astype(np.float32)


def decode(codes: np.ndarray, scale: np.ndarray, top: int) -> np.ndarray:
    """The fp32 numbers (m, or the root of v) that codes and scales stand for."""
    q = _blocks(codes).astype(np.float32)
    unit = scale.astype(np.float32) * F32(1.0 / (top * top))
    with np.errstate(all="ignore"):
        return ((q * np.abs(q)) * unit[:, None]).reshape(-1)[:codes.size]


def roots(v: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        return np.sqrt(v.astype(np.float32))


def step(grad, grad_dtype, grad_scale, master, m, v, hp, out_dtype):
    """One step of a tensor whose moments are (codes, scale) pairs: (master, m, v, out), m and v as pairs.
    The update is the full-width one on the moments' values."""
    from .adam import sharded_step
    root = decode(*v, 255)
    p, m32, v32, out = sharded_step([grad], grad_dtype, grad_scale, master, decode(*m, 127), root * root, hp, out_dtype)
    return p, encode(m32, 127), encode(roots(v32), 255), out
