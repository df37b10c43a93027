"""CPU oracle for the operators of a mixture-of-experts block.

TEST INFRASTRUCTURE ONLY (see ``oracle/gemm.py``). The CUDA library never
calls it and shares no code with it.

Everything is float64 numpy on the exact values given, not rounded to any
output type (except where a definition says that a value is held rounded: the
norm's h). The definitions are those of the C interface's comments:

* ``rms_norm``: r = (mean_j h_j^2 + eps)^-1/2, y = h r w;
  ``rms_norm_grad``: dx = r (g - xhat mean(g xhat)) + dh with g = dy w,
  xhat = h r, and dw = sum over rows of dy xhat
* ``scores``: softmax or sigmoid of a row of logits, 0 where the logit is -inf
* ``keys``: score + bias, -inf for experts that are out (logit -inf, or outside
  the best groups; a group's key is the sum of its two largest keys)
* ``route_weights`` / ``route_grad``: weights of a given choice, and the
  gradient of sum(dweights * weights) with respect to the logits
* ``order``: the stable counting sort of the (token, expert) pairs by expert
* ``grouped`` / ``grouped_wgrad``: the ragged products, group by group, each
  also with the sum of absolute products (the error scale S of oracle/check.py)
* ``combine`` / ``combine_grad``
"""

from __future__ import annotations

import numpy as np


def rms_norm(h, w, eps):
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * r[:, None] * w, r


def rms_norm_grad(dy, h, w, r, dh=None):
    dy, h, w, r = (np.asarray(x, np.float64) for x in (dy, h, w, r))
    xhat, g = h * r[:, None], dy * w
    dx = r[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return (dx if dh is None else dx + np.asarray(dh, np.float64)), (dy * xhat).sum(axis=0)


def scores(logits, kind):
    l = np.asarray(logits, np.float64)
    out = np.isneginf(l)
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            top = np.where(out, -np.inf, l).max(axis=1, keepdims=True)
            e = np.where(out, 0.0, np.exp(l - np.where(np.isneginf(top), 0.0, top)))
            z = e.sum(axis=1, keepdims=True)
            s = e / np.where(z == 0, 1.0, z)
    return np.where(out, 0.0, s)


def keys(logits, kind, bias=None, groups=1, kept=1):
    l = np.asarray(logits, np.float64)
    key = scores(l, kind) + (0.0 if bias is None else np.asarray(bias, np.float64))
    key = np.where(np.isneginf(l), -np.inf, key)
    if groups > 1:
        t, e = key.shape
        per = e // groups
        g = np.sort(key.reshape(t, groups, per), axis=2)[:, :, -2:].sum(axis=2)
        best = np.argsort(-g, axis=1, kind="stable")[:, :kept]
        keep = np.zeros((t, groups), bool)
        np.put_along_axis(keep, best, True, axis=1)
        key = np.where(np.repeat(keep, per, axis=1), key, -np.inf)
    return key


def choose(key, k):
    """The k largest keys of each row in descending order, ties to the lowest index; -1 where none is left."""
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(key, ids, 1) == -np.inf, -1, ids)


def route_weights(logits, ids, kind, renormalize=True, scale=1.0):
    s = scores(logits, kind)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renormalize:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    return w * scale


def route_grad(dweights, logits, ids, kind, renormalize=True, scale=1.0):
    s = scores(logits, kind)
    there = ids >= 0
    c = np.where(there, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    d = np.where(there, np.asarray(dweights, np.float64) * scale, 0.0)
    if renormalize:
        total = c.sum(axis=1, keepdims=True) + 1e-20
        d = np.where(there, d / total - (d * c).sum(axis=1, keepdims=True) / total ** 2, 0.0)
    ds = np.zeros_like(s)
    for t, j in zip(*np.nonzero(there)):
        ds[t, ids[t, j]] += d[t, j]
    if kind == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))


def order(ids, experts):
    """(slots, rows, offsets) of T x k expert numbers (-1: none)."""
    ids = np.asarray(ids)
    slots = np.full(ids.shape, -1, np.int64)
    rows = np.full(ids.size, -1, np.int64)
    offsets = [0]
    for e in range(experts):
        at = offsets[-1]
        for t, j in np.argwhere(ids == e):
            slots[t, j], rows[at] = at, t
            at += 1
        offsets.append(at)
    return slots, rows, np.array(offsets)


def grouped(a, w, offsets, rows=None, layout=0):
    """C and S of each slot (zeros past the last group); w: experts x K x N (layout 0) or experts x N x K."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    if layout == 1:
        w = np.swapaxes(w, 1, 2)
    n = len(a) if rows is None else len(rows)
    c, s = np.zeros((n, w.shape[2])), np.zeros((n, w.shape[2]))
    for e in range(len(w)):
        for i in range(offsets[e], offsets[e + 1]):
            x = a[i if rows is None else rows[i]]
            c[i], s[i] = x @ w[e], np.abs(x) @ np.abs(w[e])
    return c, s


def grouped_wgrad(a, dc, offsets, rows=None, layout=0):
    """dW and S of each expert."""
    a, dc = np.asarray(a, np.float64), np.asarray(dc, np.float64)
    dw, s = [], []
    for e in range(len(offsets) - 1):
        sl = slice(offsets[e], offsets[e + 1])
        x = a[sl] if rows is None else a[np.asarray(rows)[sl]]
        d = dc[sl]
        m, ms = x.T @ d, np.abs(x).T @ np.abs(d)
        dw.append(m.T if layout == 1 else m)
        s.append(ms.T if layout == 1 else ms)
    return np.stack(dw), np.stack(s)


def combine(z, slots, weights=None, residual=None):
    """y and the sum of its terms' absolute values."""
    z = np.asarray(z, np.float64)
    w = np.ones(slots.shape) if weights is None else np.asarray(weights, np.float64)
    y = np.zeros((len(slots), z.shape[1])) if residual is None else np.asarray(residual, np.float64).copy()
    s = np.abs(y)
    for t, j in np.argwhere(slots >= 0):
        y[t] += w[t, j] * z[slots[t, j]]
        s[t] += np.abs(w[t, j] * z[slots[t, j]])
    return y, s


def combine_grad(dy, z, slots, weights=None):
    dy, z = np.asarray(dy, np.float64), np.asarray(z, np.float64)
    w = np.ones(slots.shape) if weights is None else np.asarray(weights, np.float64)
    dz, dw = np.zeros_like(z), np.zeros(slots.shape)
    for t, j in np.argwhere(slots >= 0):
        dz[slots[t, j]] = w[t, j] * dy[t]
        dw[t, j] = dy[t] @ z[slots[t, j]]
    return dz, dw
