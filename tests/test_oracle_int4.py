"""The oracle of the integer 4-bit weights and of the token permutation against brute force, and its gradients
against differences. CPU only."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import int4, permute


def _rne(f: Fraction) -> int:
    n = f.numerator // f.denominator
    r = f - n
    if r > Fraction(1, 2) or (r == Fraction(1, 2) and n % 2):
        n += 1
    return n


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_quantize_by_fractions(symmetric, t):
    rng = np.random.default_rng(3)
    w = np.float32(rng.standard_normal((9, 96)) * 0.02)
    w[0] = 0.0
    w[1, :] = np.float32(np.arange(96) % 31 - 15) * np.float32(0.5)     # halves of a step: ties
    w[1, 5] = 7.5
    w[2] = np.abs(w[2]) + 1                                             # one-sided groups
    w[3] = -np.abs(w[3]) - 1
    w[4] *= np.float32(1e-9)                                            # a scale that f16 rounds to zero
    w[5] *= np.float32(1e9)                                             # a scale beyond f16
    q, s, z = int4.quantize(w, 64, symmetric, t)                        # the second group is half a group
    for n in range(9):
        for g, c in enumerate((slice(0, 64), slice(64, 96))):
            v = [Fraction(float(x)) for x in w[n, c]]
            tt = torch.bfloat16 if t == "bf16" else torch.float16
            lo, hi = min(v + [Fraction(0)]), max(v + [Fraction(0)])
            exact = max(hi, -lo) / 7 if symmetric else (hi - lo) / 15
            want = min(float(torch.tensor(float(exact), dtype=torch.float64).float().to(tt)), torch.finfo(tt).max)
            assert s[n, g] == want
            if want == 0:
                assert (q[n, c] == z[n, g]).all() and z[n, g] == (8 if symmetric else 0)
                continue
            S = Fraction(want)
            Z = 8 if symmetric else min(max(_rne(-lo / S), 0), 15)
            assert z[n, g] == Z
            assert [min(max(_rne(x / S) + Z, 0), 15) for x in v] == q[n, c].tolist()


def test_pack_and_decode():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (3, 64))
    codes = int4.pack(q)
    assert codes[1, 7] == q[1, 14] | q[1, 15] << 4 and np.array_equal(int4.unpack(codes), q)
    s, z = rng.random((3, 2)), rng.integers(0, 256, (3, 2))
    W = int4.dequantize(q, s, z, 32)
    assert W[2, 33] == (q[2, 33] - z[2, 1]) * s[2, 1]
    x = rng.standard_normal((2, 64))
    Y, B = int4.product(x, q, s, z, 32)
    assert np.allclose(Y[1, 2], sum(x[1, k] * W[2, k] for k in range(64)), rtol=1e-12)
    assert (np.abs(Y) <= B).all()


def test_product_error_covers_an_f32_evaluation():
    """s * (sum x q - z sum x) in float32, span by span, as badly ordered as the bound allows."""
    rng = np.random.default_rng(1)
    for K, group in ((512, 128), (2080, 64), (5120, 5120)):
        q, groups = rng.integers(0, 16, (8, K)), -(-K // group)
        s = np.float32(rng.random((8, groups)) * 0.01)
        z = rng.integers(0, 16, (8, groups))
        x = np.float32(rng.standard_normal((2, K)))
        Y, B = int4.product(x.astype(np.float64), q, s, z, group)
        got = np.zeros((2, 8), np.float32)
        span = 128 if group % 128 == 0 else 32
        for k0 in range(0, K, span):
            g = k0 // group
            a, b = np.zeros((2, 8), np.float32), np.zeros((2, 1), np.float32)
            for k in range(k0, min(K, k0 + span)):
                a += x[:, k, None] * np.float32(q[:, k])
                b += x[:, k, None]
            got += s[:, g] * (a - np.float32(z[:, g]) * b)
        err = np.abs(got - Y) / int4.product_error(B, K, group)
        assert 1e-4 < err.max() <= 1.0


def _differences(f, x, step=1e-3):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        p, m = x.copy(), x.copy()
        p[i] += step
        m[i] -= step
        g[i] = (f(p) - f(m)) / (2 * step)
    return g


def test_permutation_gradients_by_differences():
    """scatter and gather are each other's gradient, and the weights' gradient of both is the dot product."""
    rng = np.random.default_rng(2)
    T, k, D, R = 3, 2, 4, 5
    row_of = np.array([4, 0, -1, 2, 3, 9])
    w = rng.random((T, k))
    X, G = rng.standard_normal((T, D)), rng.standard_normal((R, D))
    zero = np.zeros((R, D))

    def permuted(X, w):
        return (permute.scatter(X, row_of, w, R, zero) * G).sum()
    assert np.allclose(_differences(lambda v: permuted(v, w), X), permute.gather(G, row_of, w, T)[0], atol=1e-9)
    assert np.allclose(_differences(lambda v: permuted(X, v), w), permute.dots(X, G, row_of)[0], atol=1e-9)
    Y, g = rng.standard_normal((R, D)), rng.standard_normal((T, D))

    def back(Y, w):
        return (permute.gather(Y, row_of, w, T)[0] * g).sum()
    assert np.allclose(_differences(lambda v: back(v, w), Y), permute.scatter(g, row_of, w, R, zero), atol=1e-9)
    assert np.allclose(_differences(lambda v: back(Y, v), w), permute.dots(g, Y, row_of)[0], atol=1e-9)
