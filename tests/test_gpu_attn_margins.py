"""The outputs of the 4-bit cache's calls, the cache itself and the attention's workspace between margins of marked
elements: no call writes outside them, and none leaves an element of an output unwritten."""
import numpy as np
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn
from attn_util import TYPES, Batch
from test_gpu_margins import Margins

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("algo", [ssn.ALGO_STREAM, ssn.ALGO_MFMA], ids=["stream", "tile"])
@pytest.mark.parametrize("D,Hq,H,lens,qs", [(32, 1, 1, [1], [1]), (96, 6, 2, [70, 5, 33], [7, 0, 33]), (128, 5, 1, [3000, 17], [1, 1]),
                                            (160, 3, 3, [2500], [19]), (224, 9, 1, [40, 200], [3, 4]), (256, 4, 2, [9001], [2]),
                                            (64, 17, 1, [5000, 4000], [5, 1])])
def test_attention(D, Hq, H, lens, qs, algo):
    """Outputs and a workspace of the very size asked for; a workspace that held something, and one that held zeros."""
    B = Batch(lens, qs, Hq, H, D, 16)
    T = sum(qs)
    for t in (torch.bfloat16, torch.float32):
        m = Margins()
        out, lse = m.tensor((T, Hq, D), t), m.tensor((T, Hq), torch.float32)
        size = ssn.lib().attn_kv_nvfp4_workspace_bytes(len(lens), Hq, H, D, max(qs), B.table.shape[1] * 16)
        B.call(algo=algo, out=out, lse=lse, workspace=m.tensor((size,), torch.uint8))
        assert m.whole()
        B.check(out, lse, out_type="f32" if t is torch.float32 else None)
        again, lse2, _ = B.call(algo=algo, out=torch.zeros_like(out), lse=torch.zeros_like(lse),
                                workspace=torch.zeros(size, dtype=torch.uint8, device="cuda"))
        assert torch.equal(out, again) and torch.equal(lse, lse2)          # every element written


@pytest.mark.parametrize("T,H,D,page", [(1, 1, 32, 16), (13, 3, 96, 48), (101, 2, 160, 16), (37, 1, 224, 80), (600, 5, 256, 32)])
def test_cache(T, H, D, page):
    """The cache's tensors and what is read of them; slots beyond the cache next to its last."""
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 1
    for t in TYPES.values():
        m = Margins()
        ts = torch.full((H,), 1e-3, device="cuda")
        cache = ssn.KvNvfp4(m.tensor((pages, H, page, D // 2), torch.uint8), m.tensor((pages, H, page, D // 16), torch.uint8),
                            m.tensor((pages, H, page, D // 2), torch.uint8), m.tensor((pages, H, D // 16, page), torch.uint8), ts, ts)
        K, V = (torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(t).cuda() for _ in range(2))
        slots = rng.permutation(pages * page - 1)[:T]
        slots[-1] = pages * page - 1
        if T > 2:
            slots[0], slots[1] = pages * page, -1
        slots = torch.from_numpy(slots).cuda()
        ssn.kv_nvfp4_append(K, V, slots, cache)
        Kr, Vr = m.tensor((T, H, D), t), m.tensor((T, H, D), t)
        ssn.kv_nvfp4_read(slots, cache, K=Kr, V=Vr)
        assert m.whole()
        again = ssn.kv_nvfp4_read(slots, cache, K=torch.zeros_like(Kr), V=torch.zeros_like(Vr))
        assert torch.equal(Kr, again[0]) and torch.equal(Vr, again[1])
