"""Tokens to expert order and back in float64 (test infrastructure only).

Entry f = t k + j owns row row_of[f] of the expert-ordered rows; outside [0, R) it has none.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24


def scatter(A, row_of, w, R, B0):
    """B0 [R, D] with B[row_of[f]] = w[f] A[t] written over it."""
    T = A.shape[0]
    B = np.array(B0, np.float64)
    k = row_of.size // T if T else 1
    for f, r in enumerate(row_of):
        if 0 <= r < R:
            B[r] = (1.0 if w is None else np.float64(w.reshape(-1)[f])) * A[f // k]
    return B


def gather(B, row_of, w, T):
    """(sum_j w[f] B[row_of[f]], the same of magnitudes)."""
    R, D = B.shape
    k = row_of.size // T if T else 1
    out, mag = np.zeros((T, D)), np.zeros((T, D))
    for f, r in enumerate(row_of):
        if 0 <= r < R:
            v = (1.0 if w is None else np.float64(w.reshape(-1)[f])) * B[r]
            out[f // k] += v
            mag[f // k] += np.abs(v)
    return out, mag


def dots(A, B, row_of):
    """(<A[t], B[row_of[f]]> [T, k], the same of magnitudes)."""
    T = A.shape[0]
    k = row_of.size // T if T else 1
    out, mag = np.zeros(row_of.size), np.zeros(row_of.size)
    for f, r in enumerate(row_of):
        if 0 <= r < B.shape[0]:
            out[f] = A[f // k] @ B[r]
            mag[f] = np.abs(A[f // k]) @ np.abs(B[r])
    return out.reshape(T, k), mag.reshape(T, k)


def gather_error(mag, k):
    """k products and k additions in f32."""
    return (k + 1) * U32 * mag


def dot_error(mag, D):
    """An f32 sum of D products whose additions are at most D / 64 + 64 deep."""
    return (D / 64 + 64) * U32 * mag
