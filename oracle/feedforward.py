"""CPU oracle (float64, numpy) of the feed-forward operators: layer norm and the
gated product with their gradients, and 8-bit matrices with a scale for each
block of 128. Written from the definitions, row by row of the formulas.

TEST INFRASTRUCTURE ONLY (see ``oracle/gemm.py``).
"""

from __future__ import annotations

import math

import numpy as np
from scipy.special import erf, expit

BLOCK = 128


def layer_norm(h, w, b, eps):
    """(y, mean, rstd) of rows h, in float64."""
    mean = h.mean(axis=1)
    rstd = 1.0 / np.sqrt(((h - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (h - mean[:, None]) * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_grad(dy, h, w, mean, rstd, dh=None):
    """(dx, dw, db) for the statistics given."""
    xhat = (h - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * xhat).sum(axis=0), dy.sum(axis=0)


def gate(x, act):
    """(activation, its slope); ReLU's slope at 0 is 0."""
    if act == "relu":
        return np.where(x > 0, x, 0.0), (x > 0).astype(np.float64)
    if act == "silu":
        p = expit(x)
        return x * p, p + x * p * (1 - p)
    if act == "gelu":
        p = 0.5 * (1 + erf(x / math.sqrt(2)))
        return x * p, p + x * np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


# The activations' largest slopes.
LIPSCHITZ = {"silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13, "relu": 1.0}


def gated(a, w, bias, act):
    """(c, up, s) with w K x 2F: s is up's sum of absolute values."""
    up, s = a @ w, np.abs(a) @ np.abs(w)
    if bias is not None:
        up, s = up + bias, s + np.abs(bias)
    f = up.shape[1] // 2
    return gate(up[:, :f], act)[0] * up[:, f:], up, s


def gated_grad(dc, up, act):
    """dup, the gradient of [gate | value]."""
    f = up.shape[1] // 2
    y, slope = gate(up[:, :f], act)
    return np.concatenate((dc * up[:, f:] * slope, dc * y), axis=1)


def spread(scale, shape, tall):
    """Scales of blocks as one for each element of a matrix of `shape`."""
    return np.repeat(np.repeat(scale, tall, axis=0)[:shape[0]], BLOCK, axis=1)[:, :shape[1]]


def block_scales(t, tall):
    """max(max |t|, 1e-12) / 448 of each block of tall x 128."""
    r, c = t.shape
    full = np.zeros((-(-r // tall) * tall, -(-c // BLOCK) * BLOCK))
    full[:r, :c] = np.abs(t)
    top = full.reshape(full.shape[0] // tall, tall, -1, BLOCK).max(axis=(1, 3))
    return np.maximum(top, 1e-12) / 448.0


def matmul_blocks(a, b, sa, sb, b_rows):
    """(c, s): the product of the numbers that the blocks stand for, and of their absolute values."""
    x, y = a * spread(sa, a.shape, 1), b * spread(sb, b.shape, b_rows)
    return x @ y.T, np.abs(x) @ np.abs(y).T
