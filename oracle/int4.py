"""Integer 4-bit weights with group scales in float64 (test infrastructure only).

W_hat[n, k] = s[n, g] * (q[n, k] - z[n, g]), g = k // group, z = 8 where no zero points are stored. 16-bit scales
are handled as the float64 values they stand for.
"""
from __future__ import annotations

import numpy as np

from . import formats

U32 = 2.0 ** -24          # half a step of f32
HALF_STEP = {"f32": U32, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LARGEST = {"bf16": float(np.uint32(0x7F7F0000).view(np.float32)), "f16": 65504.0}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}   # half the smallest subnormal


def round16(v, t):
    """float64 -> the 16-bit type t by way of f32, at most its largest value; returned as float64."""
    f = np.minimum(np.asarray(v, np.float64), LARGEST[t]).astype(np.float32)
    if t == "f16":
        return f.astype(np.float16).astype(np.float64)
    return formats.bf16_round(f.astype(np.float64))


def nearest(w, s):
    """The whole number nearest to w / s, halves to the even one (s > 0). The float64 quotient of two values of
    at most 24 bits lies on a half-integer only where the exact one does."""
    return np.rint(np.asarray(w, np.float64) / s)


def quantize(w, group, symmetric, s_type):
    """w float [N, K] -> (q int [N, K], s float64 [N, groups], z int [N, groups])."""
    w = np.asarray(w, np.float64)
    N, K = w.shape
    groups = -(-K // group)
    q = np.zeros((N, K), np.int64)
    s, z = np.zeros((N, groups)), np.zeros((N, groups), np.int64)
    for g in range(groups):
        c = slice(g * group, min(K, (g + 1) * group))
        if symmetric:
            sg = round16(np.abs(w[:, c]).max(1) / 7.0, s_type)
            zg = np.full(N, 8.0)
        else:
            lo, hi = np.minimum(w[:, c].min(1), 0.0), np.maximum(w[:, c].max(1), 0.0)
            sg = round16((hi - lo) / 15.0, s_type)
            zg = np.where(sg > 0, np.clip(nearest(-lo, np.where(sg > 0, sg, 1.0)), 0, 15), 0.0)
        safe = np.where(sg > 0, sg, 1.0)[:, None]
        qg = np.clip(nearest(w[:, c], safe) + zg[:, None], 0, 15)
        q[:, c] = np.where(sg[:, None] > 0, qg, zg[:, None])
        s[:, g], z[:, g] = sg, zg
    return q, s, z


def pack(q):
    q = np.asarray(q, np.uint8)
    return np.ascontiguousarray(q[..., 0::2] | (q[..., 1::2] << 4))


def unpack(codes):
    out = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), np.int64)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def per_k(v, group, K):
    return np.asarray(v)[..., np.arange(K) // group]


def dequantize(q, s, z, group):
    K = q.shape[-1]
    return (q - per_k(z, group, K)) * per_k(np.asarray(s, np.float64), group, K)


def product(x, q, s, z, group):
    """(Y, B): Y = x . W_hat^T for x float64 [M, K], and B = sum |x| s (q + z), the magnitudes that an f32
    evaluation of s * (sum x q - z sum x) adds up."""
    K = q.shape[-1]
    W = dequantize(q, s, z, group)
    A = (q + per_k(z, group, K)) * per_k(np.abs(np.asarray(s, np.float64)), group, K)
    return x @ W.T, np.abs(x) @ A.T


def product_error(B, K, group):
    """What an f32 evaluation may be off by: inside a span of min(group, 128) k the sums are at most that many
    additions deep, then one more per span, and 16 for the join of partial sums and the products with z and s;
    each addition errs by at most a step (2^-23) of a magnitude that B bounds."""
    span = min(group, 128) if group % 128 == 0 else 32
    return (span + -(-K // span) + 16) * 2 * U32 * B


def rounding(Y, t):
    """Half a step of type t at Y."""
    return HALF_STEP[t] * np.abs(Y) + TINY[t]


def silu_gate(g, u, eg, eu):
    """(silu(g) u, its error) for g, u with errors eg, eu: |silu'| <= 1.0999, and the f32 evaluation errs by a few
    steps plus the exponent's own rounding, (|g| + 4) 2^-22 of the result."""
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    h = s * u
    return h, 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + (np.abs(g) + 4) * 2.0 ** -22 * np.abs(h)
