"""Attention over the 4-bit cache at the ends of its numbers' range: queries that are not finite, logits of any size,
scales whose product with s_h leaves f32's range."""
import math

import numpy as np
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn
from attn_util import HALF, Batch
from oracle import kv

pytestmark = pytest.mark.gpu

both = pytest.mark.parametrize("algo", [ssn.ALGO_STREAM, ssn.ALGO_MFMA], ids=["stream", "tile"])
BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": float("-inf")}


def write(B, b, K, V, k_scale=None):
    """Keys and values of sequence b written anew, under another scale of the keys."""
    if k_scale is not None:
        B.cache = B.cache._replace(k_tensor_scale=torch.full((B.H,), k_scale, device="cuda"))
    ssn.kv_nvfp4_append(K, V, B.dev(B.slots[b]), B.cache)


@both
@pytest.mark.parametrize("bad", list(BAD))
@pytest.mark.parametrize("D,Hq,H,lens,qs", [(128, 8, 2, [700, 40, 3], [2, 1, 5]), (64, 3, 3, [33, 1, 2], [33, 1, 3]),
                                            (256, 4, 1, [90, 60], [9, 2]), (128, 8, 1, [9001, 2500], [1, 1]),
                                            (96, 12, 1, [300], [9])])
def test_queries_that_are_not_finite(D, Hq, H, lens, qs, bad, algo):
    """Every product with an infinite or undefined query is infinite or undefined, so its softmax is undefined: NaN, also
    where all products are -infinity (here: keys above zero alone). A row that keeps no key has nothing to be undefined."""
    B = Batch(lens, qs, Hq, H, D, 16)
    g = torch.Generator(device="cuda").manual_seed(1)
    for b, S in enumerate(lens):
        K, V = (torch.randn((S, H, D), generator=g, device="cuda") for _ in range(2))
        write(B, b, K.abs() + 0.5, V)
    want, wl, _ = B.call(algo=algo, with_lse=True)
    T = sum(qs)
    Q, hit = B.Q.clone(), torch.zeros((T, Hq), dtype=torch.bool, device="cuda")
    for i in range(min(T, 6)):
        t, h = T - 1 - i, (3 * i + 1) % Hq
        Q[t, h, (7 * i) % D], hit[t, h] = BAD[bad], True
    Q[0, 0, D - 1], hit[0, 0] = BAD[bad], True
    for scale in (None, -0.125):
        if scale is not None:
            want, wl, _ = B.call(algo=algo, with_lse=True, scale=scale)
        out, lse, _ = B.call(algo=algo, Q=Q, with_lse=True, scale=scale)
        none = torch.isneginf(wl)
        assert bool(out[hit & ~none].isnan().all()) and bool(lse[hit & ~none].isnan().all())
        assert torch.equal(out[~hit | none], want[~hit | none]) and torch.equal(lse[~hit | none], wl[~hit | none])


@both
@pytest.mark.parametrize("S,D,n", [(200, 64, 2), (300, 128, 1), (77, 256, 3), (9001, 128, 1)])
@pytest.mark.parametrize("e", [-8, 10, 18, 21, 22, 23, 24, 25, 26, 27, 28, 30, 34, 40, 60, 100])
def test_logits_of_any_size(e, S, D, n, algo):
    """Logits scale q0 a with a of {1/2, 1, 2, 3, 4, 6}: from 2^18 on the largest alone is left, whatever the size.
    The terms are all alike, so what they are rounded to cancels but for its half step of f16 (2^-11); each sum of f32
    has far fewer than 2^4 steps of 2^-23 to lose here. The logarithm is one logit: its factor of three roundings, the
    product, the reference's 7 and the last product, below 2^-20 of it together; log n and its rounding where logits are small."""
    H, G = 2, 3
    B = Batch([S], [n], H * G, H, D, 16)
    rng = np.random.default_rng([S, D])
    a = rng.choice([1.0, 2.0, 3.0, 4.0], (S, H))
    a[rng.permutation(S - n)[:3]], a[S - n - 5:S - n - 3], a[3] = 6.0, 0.5, 0.5
    K = torch.zeros((S, H, D), device="cuda")
    K[:, :, 0], K[:, :, 1] = torch.from_numpy(a).cuda() / 8, 6.0 / 8        # the second makes each block's scale 1
    V = torch.from_numpy(rng.standard_normal((S, H, D)).astype(np.float32)).cuda()
    write(B, 0, K, V, 1 / 8)
    k, v = B.values(0)
    assert np.array_equal(k[:, :, 0], a / 8)
    B.Q.zero_()
    q0 = np.array([1.0, -1.3828125, 1.9921875, -1.0, 1.0078125, -1.9921875]) * 2.0 ** e
    B.Q[:, :, 0] = torch.from_numpy(q0).to(B.Q.dtype)
    for scale in (D ** -0.5, 0.3):
        out, lse, _ = B.call(algo=algo, with_lse=True, scale=scale, out_dtype=torch.float32)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        if e < 18:
            B.check(out, lse, scale=float(np.float32(scale)), out_type="f32")
            continue
        for i in range(n):
            for h in range(H * G):
                z = float(np.float32(scale)) * q0[h] * k[:S - n + i + 1, h // G, 0]
                top = np.nonzero(z == z.max())[0]
                vs = v[top, h // G]
                tol = np.abs(vs).mean(0) * (2.0 ** -11 + 2.0 ** -19) + 2.0 ** -23 * np.abs(vs.mean(0))
                assert np.all(np.abs(got[i, h] - vs.mean(0)) <= tol), (i, h)
                assert abs(gl[i, h] - (z.max() + math.log(len(top)))) <= 2.0 ** -20 * abs(z.max()) + 2.0 ** -18, (i, h)


@both
@pytest.mark.parametrize("S,D", [(400, 64), (400, 128), (9001, 128), (333, 256)])
def test_small_logits_behind_huge_ones(S, D, algo):
    """The first keys' logits are some -2^27, those of the later ones a few units apart: the later are weighed as if they
    stood alone."""
    H, G, n, first = 2, 2, 2, 150
    B = Batch([S], [n], H * G, H, D, 16)
    g = torch.Generator(device="cuda").manual_seed(3)
    K, V = (torch.randn((S, H, D), generator=g, device="cuda") for _ in range(2))
    K[:, :, 0] = 0
    K[:first, :, 0] = 6.0
    write(B, 0, K, V, 1.0)
    B.Q.copy_(torch.randint(-8, 9, B.Q.shape, generator=g, device="cuda").float() / 64)
    B.Q[:, :, 0] = -2.0 ** 20
    out, lse, _ = B.call(algo=algo, with_lse=True, scale=16.0, out_dtype=torch.float32)
    keep = kv.keeps(S, n, True, 0)
    keep[:, :first] = False                            # e^(-2^27) is 0
    k, v = B.values(0)
    assert np.all(k[first:, :, 0] == 0)
    want, wl, tol, lt = kv.attention(B.Q.double().cpu().numpy(), k, v, 16.0, keep, HALF["f32"])
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= lt)


@both
@pytest.mark.parametrize("scale,size,k_scale,spread", [(1e-38, 3e38, 1.3e-5, 0.03), (3e38, 1e-38, 4.0, 0.1), (-3e38, 3e-38, 4.0, 0.1),
                                                       (1e-30, 1e33, 1e-6, 0.001), (1e-20, 1e36, 1e-20, 3e-18)])
def test_scales_and_queries_that_meet_in_the_middle(scale, size, k_scale, spread, algo):
    """The product of scale and s_h lies beyond f32's range, or among its subnormals, the logits do not."""
    B = Batch([200, 60], [2, 3], 4, 2, 64, 16)
    g = torch.Generator(device="cuda").manual_seed(5)
    for b, S in enumerate(B.lens):
        K, V = (torch.randn((S, 2, 64), generator=g, device="cuda") for _ in range(2))
        write(B, b, K * spread, V, k_scale)
    B.Q.copy_(torch.randn(B.Q.shape, generator=g, device="cuda").clamp(-1, 1) * size)
    assert bool(B.Q.isfinite().all())
    out, lse, _ = B.call(algo=algo, scale=scale, with_lse=True, out_dtype=torch.float32)
    B.check(out, lse, scale=float(np.float32(scale)), out_type="f32")


@both
@pytest.mark.parametrize("scale,size", [(1.0, 3e38), (-1.0, 3e38), (3e38, 100.0), (3e38, 3e38)])
def test_logits_beyond_f32(scale, size, algo):
    """A row whose |scale| s_h max|Q| log2(e) is 2^107 or more is undefined; the rows beside it are what they are."""
    B = Batch([150, 2], [2, 4], 4, 2, 128, 16)
    want, wl, _ = B.call(algo=algo, scale=scale, Q=B.Q * 0, with_lse=True)
    assert bool(want.isfinite().all())
    Q = B.Q * 0
    Q[1, 2, 5], Q[2, 1, 127], Q[5, 0, 0] = size, -size, size
    hit = (Q != 0).any(2)
    out, lse, _ = B.call(algo=algo, Q=Q, with_lse=True, scale=scale)
    none = torch.isneginf(wl)
    assert bool(out[hit & ~none].isnan().all()) and bool(lse[hit & ~none].isnan().all()) and bool((hit & none).any())
    assert torch.equal(out[~hit | none], want[~hit | none]) and torch.equal(lse[~hit | none], wl[~hit | none])


@both
@pytest.mark.parametrize("S,D,n", [(300, 64, 2), (9001, 128, 1), (5000, 256, 3), (200, 96, 200)])
@pytest.mark.parametrize("v_scale", [1e-37, -3e-38, 1.1e-36, 1e30])
def test_values_of_any_size(v_scale, S, D, n, algo):
    """The values' s_h over the sum of a long row lies among f32's subnormals, the result does not."""
    B = Batch([S], [n], 4, 2, D, 16)
    B.cache = B.cache._replace(v_tensor_scale=torch.tensor([1.0, 1.5], device="cuda") * v_scale)
    B.cache.v_codes.copy_(torch.randint(0, 256, B.cache.v_codes.shape, dtype=torch.uint8, device="cuda") & 0x77)
    B.Q[:, 0] = 0                                      # every key counts alike
    B.cache.v_scales.fill_(0x70)                       # 128
    out, lse, _ = B.call(algo=algo, with_lse=True, out_dtype=torch.float32)
    k, v = B.values(0)
    up = 2.0 ** -math.frexp(v_scale)[1]                # the bound is of values some way above 1e-30
    want, wl, tol, lt = kv.attention(B.Q.double().cpu().numpy(), k, v * up, D ** -0.5, kv.keeps(S, n, True, 0), HALF["f32"])
    assert np.all(np.abs(out.double().cpu().numpy() * up - want) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= lt)


@both
@pytest.mark.parametrize("size,scale", [(6e-8, 2e6), (1e-6, 1e5), (6e4, 1e-5), (6e4, 1e6), (6e4, 1e25)])
def test_half_queries_from_end_to_end(size, scale, algo):
    """f16 queries among the subnormals and next to the largest, with one row of an infinity and one of NaN."""
    B = Batch([130, 40, 2100], [2, 1, 1], 4, 2, 96, 16, x="f16")
    Q = (B.Q.float().clamp(-1, 1) * size).half()
    assert bool(Q.isfinite().all()) and bool(Q.count_nonzero())
    want, wl, _ = B.call(algo=algo, Q=Q, scale=scale, with_lse=True)
    assert bool(want.isfinite().all()) and bool(wl.isfinite().all())
    if abs(size * scale) < 1e6:                        # beyond, one key alone is left, and the bound says nothing of it
        B.check(want, wl, Q=Q, scale=float(np.float32(scale)))
    else:
        top = [np.einsum("hd,shd->hs", Q[t].double().cpu().numpy(), B.values(b)[0].repeat(2, 1))[:, :S].argmax(1)
               for t, b, S in ((1, 0, 130), (2, 1, 40), (3, 2, 2100))]
        for i, (t, b) in enumerate(((1, 0), (2, 1), (3, 2))):
            v = B.values(b)[1].repeat(2, 1)[top[i], np.arange(4)]
            assert np.all(np.abs(want[t].double().cpu().numpy() - v) <= np.abs(v) * (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -19))
    bad = Q.clone()
    bad[1, 2, 95], bad[3, 0, 1] = float("-inf"), float("nan")
    out, lse, _ = B.call(algo=algo, Q=bad, scale=scale, with_lse=True)
    hit = ~bad.isfinite().all(2)
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])
