"""A cache of keys and values in NVFP4 and attention over it (oracle).

A token's D values of one head are quantised as a row of ``quant.quantize`` with the head's tensor scale given; a
cached value is E2M1(code) * E4M3(scale) * s_h. Attention is the softmax over the keys that a query keeps, in float64,
sequence by sequence and head by head. The pages define neither the layout nor the attention, so "parity unpinned": the
layout is this library's, the attention the textbook's.
"""
from __future__ import annotations

import math

import numpy as np

from .formats import e2m1_decode, e4m3_decode
from .quant import quantize, unpack_nibbles


def quantize_tokens(x: np.ndarray, ts: np.ndarray):
    """x [T, H, D] (float32), ts [H] -> (codes u8 [T, H, D/2], scales u8 [T, H, D/16])."""
    T, H, D = x.shape
    codes, scales = np.zeros((T, H, D // 2), np.uint8), np.zeros((T, H, D // 16), np.uint8)
    for h in range(H):
        codes[:, h], scales[:, h], _ = quantize(np.ascontiguousarray(x[:, h]), tensor_scale_in=np.float32(ts[h]))
    return codes, scales


def dequantize_tokens(codes: np.ndarray, scales: np.ndarray, ts: np.ndarray) -> np.ndarray:
    """The values that codes [T, H, D/2] and scales [T, H, D/16] stand for, [T, H, D] in float64."""
    T, H, Dh = codes.shape
    v = e2m1_decode(unpack_nibbles(codes.reshape(T * H, Dh))).reshape(T, H, 2 * Dh)
    return v * np.repeat(e4m3_decode(scales), 16, axis=2) * np.asarray(ts, np.float64)[None, :, None]


def gather(k_codes, k_scales, v_codes, v_scales, slots, page):
    """Codes and scales of the tokens at `slots`, tokens first: (k_codes, k_scales, v_codes, v_scales)."""
    p, o = np.asarray(slots) // page, np.asarray(slots) % page
    return k_codes[p, :, o], k_scales[p, :, o], v_codes[p, :, o], v_scales[p, :, :, o]


def keeps(S: int, n: int, causal: bool, window: int) -> np.ndarray:
    """[n, S]: whether query i (at position S - n + i) keeps key j."""
    pos, j = np.arange(S - n, S)[:, None], np.arange(S)[None, :]
    keep = np.ones((n, S), bool)
    if causal:
        keep = j <= pos
        if window:
            keep = keep & (j > pos - window)
    return keep


def attention(q, k, v, scale, keep, out_eps=0.0):
    """One sequence: q [n, Hq, D], k and v [S, H, D], keep [n, S], all float64 -> (out [n, Hq, D], lse [n, Hq], and how
    far a result may lie from each).

    The bounds count an f32 evaluation whose softmax terms are rounded to f16 before they multiply v. With y a logit
    in powers of two: the sum of D products is off by at most D + 8 steps (2^-23, whatever the order and the rounding
    of a step) of sum |q k|, the factor and the subtraction of the reference by 8 steps of |y| and of the reference,
    so a term is off by a factor of at most 1 + e, e = ln 2 dy + 2^-21 (the exponential's own error). Numerator and
    denominator carry that; the numerator also half a step of f16 (2^-11 of a term, or 2^-25 where a term lies below
    f16's normal range, the largest term of a row being 2^7 at least) and both the additions, a step (2^-23) for each
    key. out_eps: half a step of the result's type relative to the result."""
    n, Hq, D = q.shape
    S, H, _ = k.shape
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    tol, ltol = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    step = 2.0 ** -23
    for h in range(Hq):
        K, V = k[:, h // (Hq // H)], v[:, h // (Hq // H)]
        z = scale * (q[:, h] @ K.T)
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(K).T) / math.log(2)
        for i in range(n):
            j = np.nonzero(keep[i])[0]
            if not j.size:
                continue
            top = z[i, j].max()
            e = np.exp(z[i, j] - top)
            w = e / e.sum()
            out[i, h] = w @ V[j]
            lse[i, h] = top + math.log(e.sum())
            dy = step * ((D + 8) * mag[i, j].max() + 16 * np.abs(z[i, j]).max() / math.log(2) + 16)
            rel = math.log(2) * dy + 2.0 ** -21 + step * j.size
            a = w @ np.abs(V[j])
            tol[i, h] = (a * (2 * rel + 2.0 ** -11) + j.size * 2.0 ** -32 * np.abs(V[j]).max(0)) * (1 + rel) \
                + out_eps * np.abs(out[i, h]) * 1.01 + 1e-30
            ltol[i, h] = 1.01 * rel + 4 * step * abs(lse[i, h]) + 2.0 ** -21
    return out, lse, tol, ltol
