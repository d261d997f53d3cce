"""Every output of the integer 4-bit and permutation calls lies between two margins of marked elements in one
allocation, at sizes that leave remainders of tiles, vectors and waves: no call writes outside its output, and
none leaves an element of it unwritten."""
import numpy as np
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MARK = 0xA5


class Margins:
    """Tensors whose bytes, and 4096 on either side of them, hold MARK; 16-byte aligned at any size."""
    PAD = 4096

    def __init__(self):
        self.made = []

    def tensor(self, shape, dtype):
        size = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        flat = torch.full((size + 2 * self.PAD,), MARK, dtype=torch.uint8, device="cuda")
        self.made.append(flat)
        return flat[self.PAD:self.PAD + size].view(dtype).view(shape)

    def whole(self):
        return all(bool((f[:self.PAD] == MARK).all()) and bool((f[len(f) - self.PAD:] == MARK).all()) for f in self.made)


def marked(t):
    """Rows whose every byte is MARK."""
    return (t.contiguous().view(torch.uint8) == MARK).all(1)


def weights(rng, lead, K, group):
    groups = -(-K // group)
    return (torch.from_numpy(rng.integers(0, 256, (*lead, K // 2)).astype(np.uint8)).cuda(),
            torch.from_numpy(rng.random((*lead, groups)) * 0.01 + 1e-3).bfloat16().cuda(),
            torch.from_numpy(rng.integers(0, 16, (*lead, groups)).astype(np.uint8)).cuda())


# up to 4, 8 and 16 rows in registers; more rows, or a longer K, by tiles of 16, 32 and 64 rows
@pytest.mark.parametrize("M", [1, 3, 4, 5, 8, 9, 15, 17, 31, 33, 50, 65])
def test_gemv(M):
    rng = np.random.default_rng(M)
    X = torch.from_numpy(rng.standard_normal((M, 160))).bfloat16().cuda()
    for N in (1, 2, 15, 17, 31, 33, 63, 65, 255, 4097):
        w = weights(rng, (N,), 160, 64)
        for t in TYPES.values():
            m = Margins()
            Y = m.tensor((M, N), t)
            ssn.gemv_int4(X, *w, group=64, Y=Y)
            assert m.whole(), (N, t)
            again = ssn.gemv_int4(X, *w, group=64, Y=torch.zeros_like(Y))[0]
            assert torch.equal(Y, again), (N, t)          # every element written


@pytest.mark.parametrize("M,N,K", [(9, 16405, 96), (16, 16399, 1056), (13, 12345, 160), (29, 12345, 160), (61, 13801, 160),
                                   (130, 12289, 160), (2, 33, 8224), (5, 70, 16416)])
def test_gemv_large(M, N, K):
    """9 to 16 rows over many weight rows, every width of tile, rows beyond 8192."""
    rng = np.random.default_rng(M + N)
    w = weights(rng, (N,), K, 128)
    X = torch.from_numpy(rng.standard_normal((M, K))).half().cuda()
    m = Margins()
    Y = m.tensor((M, N), torch.float16)
    ssn.gemv_int4(X, *w, Y=Y)
    assert m.whole()
    assert torch.equal(Y, ssn.gemv_int4(X, *w, Y=torch.zeros_like(Y))[0])


@pytest.mark.parametrize("counts", [[1], [3], [2, 0, 19, 1], [9] * 5, [0, 33, 0, 17, 1, 64]])
@pytest.mark.parametrize("K", [160, 8224])
def test_grouped(counts, K):
    """The experts' rows end at the last row of Y, or before it: the rows behind keep what they held."""
    rng = np.random.default_rng(K)
    E, used = len(counts), sum(counts)
    off = torch.from_numpy(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)).cuda()
    for N in (2, 30, 34, 66, 130):
        w = weights(rng, (E, N), K, 96)
        for R in (used, used + 2):
            X = torch.from_numpy(rng.standard_normal((R, K))).bfloat16().cuda()
            for epilogue, No in ((ssn.EPI_NONE, N), (ssn.EPI_SILU_GATE, N // 2)):
                m = Margins()
                Y = m.tensor((R, No), torch.bfloat16)
                args = dict(group=96, epilogue=epilogue)
                ssn.moe_grouped_gemv_int4(X, None, off, R, *w, Y=Y, **args)
                assert m.whole() and bool(marked(Y[used:]).all()), (N, R, epilogue)
                again = ssn.moe_grouped_gemv_int4(X, None, off, R, *w, Y=torch.zeros_like(Y), **args)[0]
                assert torch.equal(Y[:used], again[:used]), (N, R, epilogue)


@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (3, 96, 32), (5, 160, 64), (33, 224, 96), (7, 2080, 128), (3, 992, 256),
                                       (5, 1056, 512), (3, 4128, 2048), (3, 12320, 4096), (2, 9248, 9248), (255, 2080, 64)])
@pytest.mark.parametrize("symmetric", [False, True])
def test_quantize_and_dequantize(N, K, group, symmetric):
    rng = np.random.default_rng(K)
    W = torch.from_numpy(np.float32(rng.standard_normal((N, K)))).cuda()
    groups = -(-K // group)
    for t in TYPES.values():
        m = Margins()
        codes, scales = m.tensor((N, K // 2), torch.uint8), m.tensor((N, groups), torch.bfloat16)
        zeros = None if symmetric else m.tensor((N, groups), torch.uint8)
        ssn.int4_quantize(W.to(t), group=group, symmetric=symmetric, codes=codes, scales=scales, zeros=zeros)
        assert m.whole()
        fresh = [None if o is None else torch.zeros_like(o) for o in (codes, scales, zeros)]
        for a, b in zip((codes, scales, zeros), ssn.int4_quantize(W.to(t), group, symmetric, torch.bfloat16, *fresh)):
            assert a is None or torch.equal(a, b)
        out = m.tensor((N, K), t)
        ssn.int4_dequantize(codes, scales, zeros, group=group, out=out)
        assert m.whole()
        assert torch.equal(out, ssn.int4_dequantize(codes, scales, zeros, group=group, out=torch.zeros_like(out)))


@pytest.mark.parametrize("D", [1, 2, 3, 5, 7, 8, 9, 63, 65, 255, 513, 1001, 1025, 2049, 4100])
@pytest.mark.parametrize("t,out_t", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_permutation(D, t, out_t):
    """Rows that no entry owns, the first and the last among them, keep what they held."""
    rng = np.random.default_rng(D)
    T, k, R = 7, 5, 40
    place = 1 + rng.permutation(R - 2)[:T * k]
    place[3] = -1
    row_of = torch.from_numpy(place.astype(np.int32)).cuda()
    owned = torch.zeros(R, dtype=torch.bool, device="cuda")
    owned[row_of[row_of >= 0].long()] = True
    w = torch.rand((T, k), device="cuda") + 0.5
    X, G = torch.randn((T, D), device="cuda").to(TYPES[t]), torch.randn((R, D), device="cuda").to(TYPES[t])
    dout = torch.randn((T, D), device="cuda").to(TYPES[out_t])
    m = Margins()

    def calls(make):
        rows = [make((R, D), TYPES[t]) for _ in range(3)]
        dX, out, dw = make((T, D), TYPES[t]), make((T, D), TYPES[out_t]), [make((T, k), torch.float32) for _ in range(2)]
        ssn.moe_permute(X, row_of, w, R=R, Xp=rows[0])
        ssn.moe_permute_backward(G, row_of, T, w, X=X, dX=dX, dweights=dw[0])
        ssn.moe_unpermute(G, row_of, T, w, out=out)
        ssn.moe_unpermute_backward(dout, row_of, R, w, Yp=G, dYp=rows[1], dweights=dw[1])
        ssn.moe_unpermute_backward(dout, row_of, R, w, y_dtype=TYPES[t], dYp=rows[2])
        return rows, (dX, out, *dw)

    rows, tokens = calls(m.tensor)
    assert m.whole()
    rows2, tokens2 = calls(lambda shape, dtype: torch.zeros(shape, dtype=dtype, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(tokens, tokens2))
    for a, b in zip(rows, rows2):
        assert bool(marked(a[~owned]).all()) and torch.equal(a[owned], b[owned]) and not bool(b[~owned].any())
