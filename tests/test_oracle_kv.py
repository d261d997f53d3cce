"""The oracle of the 4-bit cache and its attention against definitions in plain loops."""
import math

import numpy as np

from oracle import kv, quant


def test_tokens_are_rows_of_the_quantiser():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, 3, 64)).astype(np.float32)
    ts = np.float32([1e-3, 2e-3, 5e-4])
    codes, scales = kv.quantize_tokens(x, ts)
    for t in range(7):
        for h in range(3):
            c, s, _ = quant.quantize(x[t, h][None], tensor_scale_in=ts[h])
            assert np.array_equal(codes[t, h], c[0]) and np.array_equal(scales[t, h], s[0])
    d = kv.dequantize_tokens(codes, scales, ts)
    # Where a block's largest magnitude is at most 2688 s_h, S s_h is amax / 6 within E4M3's half step (2^-4), and E2M1's
    # widest half step is 1: no value is off by more than (1 + 2^-4) amax / 6. Beyond, S is 448 and values clip.
    amax = np.repeat(np.abs(x).reshape(7, 3, 4, 16).max(3), 16, axis=2)
    within = amax <= 2688 * ts[None, :, None]
    assert within.any() and np.all((np.abs(d - x) <= amax / 6 * 1.0626)[within])
    assert np.all((np.abs(d) <= 2688 * ts[None, :, None] * 1.000001))


def test_keeps():
    assert kv.keeps(3, 2, True, 0).tolist() == [[True, True, False], [True, True, True]]
    assert kv.keeps(3, 2, True, 1).tolist() == [[False, True, False], [False, False, True]]
    assert kv.keeps(2, 3, True, 0).tolist() == [[False, False], [True, False], [True, True]]
    assert kv.keeps(2, 1, False, 0).all()


def test_attention_by_loops():
    rng = np.random.default_rng(2)
    n, S, H, G, D = 3, 11, 2, 2, 8
    q, k, v = rng.standard_normal((n, H * G, D)), rng.standard_normal((S, H, D)), rng.standard_normal((S, H, D))
    keep = kv.keeps(S, n, True, 4)
    out, lse, tol, ltol = kv.attention(q, k, v, 0.3, keep)
    for i in range(n):
        for h in range(H * G):
            num, den = np.zeros(D), 0.0
            for j in range(S):
                if keep[i, j]:
                    e = math.exp(0.3 * sum(q[i, h, d] * k[j, h // G, d] for d in range(D)))
                    den += e
                    num += e * v[j, h // G]
            assert np.allclose(out[i, h], num / den, rtol=1e-12) and abs(lse[i, h] - math.log(den)) < 1e-12
    assert np.all(tol > 0) and np.all(ltol > 0)


def test_rows_without_keys():
    q, k, v = np.ones((3, 1, 4)), np.ones((1, 1, 4)), np.ones((1, 1, 4))
    out, lse, _, _ = kv.attention(q, k, v, 1.0, kv.keeps(1, 3, True, 0))
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(out[2] == 1) and lse[2, 0] == 4.0


def test_the_bound_holds_an_evaluation_that_errs():
    """Terms rounded to f16 and sums in f32, in the kernel's units (2^7 for the largest term), stay inside."""
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((2, 1, 64)) * 3, rng.standard_normal((500, 1, 64)), rng.standard_normal((500, 1, 64))
    keep = kv.keeps(500, 2, True, 0)
    out, lse, tol, ltol = kv.attention(q, k, v, 0.125, keep)
    worst = 0.0
    for i in range(2):
        y = (np.float32(0.125 / math.log(2)) * (q[i, 0].astype(np.float32) @ k[:, 0].T.astype(np.float32)))[keep[i]]
        p = np.exp2(y - y.max() + np.float32(7)).astype(np.float32)
        got = (p.astype(np.float16).astype(np.float32) @ v[keep[i], 0].astype(np.float32)) / p.sum(dtype=np.float32)
        err = np.abs(got - out[i, 0])
        assert np.all(err <= tol[i, 0])
        worst = max(worst, float((err / tol[i, 0]).max()))
    assert worst > 0.01
