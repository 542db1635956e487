"""Tokens sorted by expert and back: the order, the gathered rows, the weighted
sum and its gradients, in plain numpy and 64 bits."""

import numpy as np


def capacity(slots, experts, align):
    if align == 1:
        return slots
    rows = slots + min(experts, slots) * (align - 1)
    return -(-rows // 256) * 256


def sort(ids, experts, align, rows=None):
    """(offsets, slots, where) of ids [t][k]: expert by expert, slots ascending."""
    flat = np.asarray(ids).reshape(-1)
    n = capacity(flat.size, experts, align) if rows is None else rows
    offsets, slots, where = np.zeros(experts + 1, np.int32), np.full(n, -1, np.int32), np.full(flat.size, -1, np.int32)
    at = 0
    for e in range(experts):
        mine = np.nonzero(flat == e)[0]
        offsets[e] = at
        slots[at:at + mine.size] = mine
        where[mine] = np.arange(at, at + mine.size)
        at += -(-mine.size // align) * align
    offsets[experts] = at
    return offsets, slots, where.reshape(np.asarray(ids).shape)


def gather(x, slots, k):
    """x[slots / k], zero where there is no slot (any dtype)."""
    out = np.zeros((len(slots), x.shape[1]), x.dtype)
    out[slots >= 0] = x[slots[slots >= 0] // k]
    return out


def combine(z, where, weights=None, residual=None):
    """(sum, sum of magnitudes) in float64."""
    out, mag = np.zeros((2, len(where), z.shape[1]))
    for t, row in enumerate(where):
        for j, r in enumerate(row):
            if r >= 0:
                term = (1.0 if weights is None else float(weights[t, j])) * z[r].astype(np.float64)
                out[t] += term
                mag[t] += abs(term)
    if residual is not None:
        out += residual
        mag += abs(residual)
    return out, mag


def combine_backward(dy, z, where, weights):
    """(dz, dw, magnitudes of dw's sums) in float64; dz is zero in rows without a slot."""
    dz, dw, mag = np.zeros(z.shape), np.zeros(where.shape), np.zeros(where.shape)
    for t, row in enumerate(where):
        for j, r in enumerate(row):
            if r >= 0:
                dz[r] = float(weights[t, j]) * dy[t]
                dw[t, j] = dy[t] @ z[r].astype(np.float64)
                mag[t, j] = abs(dy[t]) @ abs(z[r].astype(np.float64))
    return dz, dw, mag
