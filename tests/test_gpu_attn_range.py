"""Attention over the 4-bit cache at the ends of its numbers' range: queries that are not finite."""
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn
from attn_util import Batch

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
