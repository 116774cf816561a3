"""Plain 64-bit references of the routed layers, for the tests (numpy)."""
from __future__ import annotations

import numpy as np


def plan(ids, groups, align, capacity=None):
    """(offsets, rows, src) by going through the pairs one after the other."""
    flat = np.asarray(ids).reshape(-1)
    kept = (flat >= 0) & (flat < groups)
    counts = np.bincount(flat[kept].astype(np.int64), minlength=groups)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    least = -(-(flat.size + min(flat.size, groups) * (align - 1)) // align) * align
    src = np.full(least if capacity is None else capacity, -1, np.int64)
    rows = np.full(flat.size, -1, np.int64)
    nxt = offsets[:-1].copy()
    for p in np.nonzero(kept)[0]:
        g = int(flat[p])
        rows[p] = nxt[g]
        src[nxt[g]] = p
        nxt[g] += 1
    return offsets, rows.reshape(np.shape(ids)), src


def combine(y, rows, weights, residual):
    """(out, sum of the terms' magnitudes)."""
    kept = rows >= 0
    part = np.where(kept[..., None], weights[..., None] * y[np.where(kept, rows, 0)], 0.0)
    return residual + part.sum(1), np.abs(residual) + np.abs(part).sum(1)


def combine_grad(dout, y, rows, src, weights):
    """(dy, dweights, sum of the magnitudes of dweights' terms)."""
    k = rows.shape[1]
    pair = np.where(src >= 0, src, 0)
    dy = np.where((src >= 0)[:, None], weights.reshape(-1)[pair][:, None] * dout[pair // k], 0.0)
    kept = rows >= 0
    terms = np.where(kept[..., None], dout[:, None] * y[np.where(kept, rows, 0)], 0.0)
    return dy, terms.sum(-1), np.abs(terms).sum(-1)


def adapters(x, A, B, ids, scale, base):
    """(y, magnitude of the terms of the low-rank part)."""
    y, size = base.copy(), np.zeros_like(base)
    for g in range(len(A)):
        t = ids == g
        y[t] += scale[g] * (x[t] @ A[g].T) @ B[g].T
        size[t] = abs(scale[g]) * (np.abs(x[t]) @ np.abs(A[g]).T) @ np.abs(B[g]).T
    return y, size


def adapters_grad(dy, x, A, B, ids, scale, dres):
    """(dx, dA, dB) and the magnitudes of their terms."""
    dx, dA, dB = dres.copy(), np.zeros_like(A), np.zeros_like(B)
    sx, sA, sB = np.zeros_like(dres), np.zeros_like(A), np.zeros_like(B)
    for g in range(len(A)):
        t = ids == g
        d = scale[g] * dy[t]
        dx[t] += d @ B[g] @ A[g]
        dA[g] = (d @ B[g]).T @ x[t]
        dB[g] = d.T @ (x[t] @ A[g].T)
        d, xa, Aa, Ba = np.abs(d), np.abs(x[t]), np.abs(A[g]), np.abs(B[g])
        sx[t], sA[g], sB[g] = d @ Ba @ Aa, (d @ Ba).T @ xa, d.T @ (xa @ Aa.T)
    return (dx, dA, dB), (sx, sA, sB)
