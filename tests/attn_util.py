"""Batches of sequences in a shuffled 4-bit cache for the attention tests, and their check against the oracle."""
import numpy as np
import torch

import structured_sparse_nvfp4_amd as ssn
from oracle import kv

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


class Batch:
    """Sequences of the given lengths and numbers of queries in a shuffled cache whose unused slots hold 0xFF (NaN
    scales) and whose unused table entries are no pages."""

    def __init__(self, lens, qs, Hq, H, D, page, seed=0, x="bf16", spread=1.0, spare=2):
        rng = np.random.default_rng([seed, D, page])
        self.lens, self.qs, self.Hq, self.H, self.D, self.page, self.x = list(lens), list(qs), Hq, H, D, page, x
        used = [-(-n // page) for n in lens]
        pages = sum(used) + spare
        ts = (rng.random((2, H)) * 1e-3 + 1e-3).astype(np.float32)
        self.cache = ssn.kv_nvfp4_empty(pages, page, D, torch.from_numpy(ts[0]).cuda(), torch.from_numpy(ts[1]).cuda())
        for t in self.cache[:4]:
            t.fill_(0xFF)
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(used + [0]) + 1), -1, np.int32)
        self.slots, at = [], 0
        for b, n in enumerate(lens):
            self.table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            j = np.arange(n)
            self.slots.append(self.table[b, j // page].astype(np.int64) * page + j % page)
        T = sum(lens)
        if T:
            slots = torch.from_numpy(np.concatenate(self.slots)).cuda()
            K, V = (torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32) * s).cuda() for s in (spread, 1.0))
            ssn.kv_nvfp4_append(K, V, slots, self.cache)
        self.Q = torch.from_numpy(rng.standard_normal((sum(qs), Hq, D)).astype(np.float32)).to(TYPES[x]).cuda()
        self.offsets = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def call(self, uniform=False, **kw):
        off = None if uniform else self.dev(self.offsets)
        kw.setdefault("max_q", max(self.qs))
        return ssn.attn_kv_nvfp4(kw.pop("Q", self.Q), self.cache, self.dev(self.table), self.dev(np.int32(self.lens)), off, **kw)

    def values(self, b):
        """Cached keys and values of sequence b in float64."""
        h = [t.cpu().numpy() for t in self.cache]
        kc, ks, vc, vs = kv.gather(*h[:4], self.slots[b], self.page)
        return kv.dequantize_tokens(kc, ks, h[4]), kv.dequantize_tokens(vc, vs, h[5])

    def check(self, out, lse=None, causal=True, window=0, scale=None, Q=None, out_type=None, seqs=None):
        torch.cuda.synchronize()
        Q = (self.Q if Q is None else Q).double().cpu().numpy()
        got = out.double().cpu().numpy()
        eps = HALF[out_type or self.x]
        for b in range(len(self.lens)) if seqs is None else seqs:
            q0, n, S = int(self.offsets[b]), self.qs[b], self.lens[b]
            k, v = self.values(b)
            want, wlse, tol, ltol = kv.attention(Q[q0:q0 + n], k, v, self.D ** -0.5 if scale is None else scale,
                                                 kv.keeps(S, n, causal, window), eps)
            bad = ~(np.abs(got[q0:q0 + n] - want) <= tol)
            assert not bad.any(), (b, np.argwhere(bad)[:3].tolist(), int(bad.sum()), got[q0:q0 + n][bad][:3], want[bad][:3], tol[bad][:3])
            if lse is not None:
                gl = lse[q0:q0 + n].double().cpu().numpy()
                none = np.isneginf(wlse)
                assert np.array_equal(np.isneginf(gl), none)
                assert np.all(np.abs(gl[~none] - wlse[~none]) <= ltol[~none])
