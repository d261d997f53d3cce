"""GPU parity of the integer 4-bit weights (quantise, dequantise, the products plain and grouped) against the
float64 oracle. Quantisation is bit-exact; products stay within the bound of their f32 evaluation plus half a
step of the output type."""
import numpy as np
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn
from oracle import int4

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def np64(t):
    return t.detach().cpu().double().numpy()


def make_weights(rng, lead, K, group, asym, s_type, wide=False):
    """(q, s, z) for the oracle and (codes, scales, zeros) on the GPU; wide: zero points over all of a byte."""
    groups = -(-K // group)
    q = rng.integers(0, 16, (*lead, K))
    scales = torch.from_numpy(rng.random((*lead, groups)) * 0.02 + 1e-3).to(TYPES[s_type])
    z = rng.integers(0, 256 if wide else 16, (*lead, groups)) if asym else np.full((*lead, groups), 8)
    zeros = torch.from_numpy(z.astype(np.uint8)).cuda() if asym else None
    return (q, np64(scales), z), (torch.from_numpy(int4.pack(q)).cuda(), scales.cuda(), zeros)


def make_x(rng, shape, x_type):
    X = torch.from_numpy(rng.standard_normal(shape)).to(TYPES[x_type])
    return np64(X), X.cuda()


# ------------------------------------------------------------------------------ quantise, dequantise
def special_weights(rng, N, K):
    w = np.float32(rng.standard_normal((N, K)) * 0.02)
    if N >= 8:
        w[0] = 0.0
        w[1] = np.float32(np.arange(K) % 31 - 15) * np.float32(0.5)          # halves of a step
        w[2], w[3] = np.abs(w[2]) + 1, -np.abs(w[3]) - 1                     # one-sided groups
        w[4] *= np.float32(1e-9)                                             # f16 scales that round to zero
        w[5] *= np.float32(1e9)                                              # f16 scales at their largest
        w[6] *= np.float32(1e-37)                                            # subnormal weights and bf16 scales
        w[7] = np.float32(rng.choice([-3e38, 3e38, 0.0], K))                 # a range beyond f32
    return w


@pytest.mark.parametrize("w_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("s_type", ["bf16", "f16"])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (9, 64, 64), (9, 256, 128), (37, 2080, 64), (9, 512, 512),
                                       (9, 1056, 96), (9, 1024, 4096), (300, 5120, 128), (9, 2048, 1024)])
def test_quantize_is_exact(N, K, group, symmetric, s_type, w_type):
    rng = np.random.default_rng(N + K)
    W = torch.from_numpy(special_weights(rng, N, K)).clamp(-6e4, 6e4) if w_type == "f16" else \
        torch.from_numpy(special_weights(rng, N, K))
    W = W.to(TYPES[w_type])
    q, s, z = int4.quantize(np64(W), group, symmetric, s_type)
    codes, scales, zeros = ssn.int4_quantize(W.cuda(), group=group, symmetric=symmetric, scale_dtype=TYPES[s_type])
    assert np.array_equal(np64(scales), s)
    if symmetric:
        assert zeros is None
    else:
        assert np.array_equal(zeros.cpu().numpy(), z)
    assert np.array_equal(codes.cpu().numpy(), int4.pack(q))


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 256, 512, 1024, 2048, 2080, 4096, 8192, 12320])
def test_quantize_close_to_halves(group, symmetric):
    """Weights at, and a few bits to either side of, the middle between two codes."""
    rng = np.random.default_rng(group)
    K = 2 * group + 32                                    # two groups and a short one
    W = (rng.integers(-15, 16, (40, K)) + 0.5) * rng.choice([1.0, 0.7], (40, 1))
    W *= 1 + rng.choice([-1.0, 0.0, 1.0], W.shape) * 2.0 ** -rng.integers(10, 25, W.shape)
    lo, hi = (-7.0, 7.0) if symmetric else (-7.0, 8.0)    # ranges whose scale is 1, or 0.7 rounded
    W = np.clip(W, lo, hi)
    W[:, ::32], W[:, 1::32] = lo, hi
    W = torch.from_numpy(np.float32(W))
    q, s, z = int4.quantize(np64(W), group, symmetric, "bf16")
    codes, scales, zeros = ssn.int4_quantize(W.cuda(), group=group, symmetric=symmetric)
    assert np.array_equal(np64(scales), s) and (symmetric or np.array_equal(zeros.cpu().numpy(), z))
    assert np.array_equal(codes.cpu().numpy(), int4.pack(q))


@pytest.mark.parametrize("out_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K,group,asym,s_type", [(1, 32, 32, True, "bf16"), (17, 2080, 64, True, "f16"),
                                                   (5, 5152, 96, False, "bf16"), (3, 256, 512, True, "f16")])
def test_dequantize(N, K, group, asym, s_type, out_type):
    rng = np.random.default_rng(K)
    (q, s, z), dev = make_weights(rng, (N,), K, group, asym, s_type, wide=True)
    W = torch.from_numpy(int4.dequantize(q, s, z, group)).float()       # at most 20 bits: exact in f32
    assert torch.equal(ssn.int4_dequantize(*dev, group=group, out_dtype=TYPES[out_type]).cpu(), W.to(TYPES[out_type]))


@pytest.mark.parametrize("out_type,N", [("f32", 6600), ("bf16", 13100), ("f16", 13100)])
def test_dequantize_beyond_the_cache(out_type, N):
    """Output of 128 MB and more, which is written past the caches: whole against f32 arithmetic on the GPU."""
    K, group = 5152, 96
    g = torch.Generator(device="cuda").manual_seed(N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand((N, -(-K // group)), generator=g, device="cuda").bfloat16()
    zeros = torch.randint(0, 256, scales.shape, generator=g, device="cuda", dtype=torch.uint8)
    got = ssn.int4_dequantize(codes, scales, zeros, group=group, out_dtype=TYPES[out_type])
    q = torch.stack((codes & 15, codes >> 4), 2).view(N, K).float()
    spread = lambda v: v.float().repeat_interleave(group, 1)[:, :K]
    assert torch.equal(got, ((q - spread(zeros)) * spread(scales)).to(TYPES[out_type]))    # at most 17 bits: exact


def test_quantize_into_given_tensors_and_back():
    rng = np.random.default_rng(5)
    W = torch.from_numpy(np.float32(rng.standard_normal((33, 320)))).cuda()
    codes = torch.zeros((33, 160), dtype=torch.uint8, device="cuda")
    s = torch.zeros((33, 5), dtype=torch.float16, device="cuda")
    z = torch.zeros((33, 5), dtype=torch.uint8, device="cuda")
    got = ssn.int4_quantize(W, group=64, codes=codes, scales=s, zeros=z)
    assert got[0] is codes and got[1] is s and got[2] is z
    back = ssn.int4_dequantize(codes, s, z, group=64)
    step = s.float().repeat_interleave(64, 1)
    # half a step, and a step where the zero point and the range's end round apart
    assert bool(((back - W).abs() <= 1.01 * step).all())


def test_any_group_beyond_the_row_is_one_group():
    """Through the C entry: up to the last multiple of 32 of its 64 bits, as a group of K."""
    rng = np.random.default_rng(7)
    for K in (32, 64, 5120):
        W = torch.from_numpy(np.float32(rng.standard_normal((9, K)))).cuda()
        codes, scales, zeros = ssn.int4_quantize(W, group=K)
        back = ssn.int4_dequantize(codes, scales, zeros, group=K)
        for group in (K + 32, 1 << 40, (1 << 63) - 32):
            got = [torch.zeros_like(t) for t in (codes, scales, zeros, back)]
            at = [t.data_ptr() for t in got]
            stream = torch.cuda.current_stream().cuda_stream
            assert ssn.lib().int4_quantize(W.data_ptr(), ssn.SSN_F32, 9, K, group, ssn.SSN_BF16, *at[:3], stream) == 0
            assert ssn.lib().int4_dequantize(at[0], at[1], ssn.SSN_BF16, at[2], 9, K, group, at[3], ssn.SSN_F32,
                                             stream) == 0
            assert all(torch.equal(a, b) for a, b in zip(got, (codes, scales, zeros, back)))


# ------------------------------------------------------------------------------ product
def check_product(got, Y, err, y_type):
    tol = err + int4.rounding(np.abs(Y) + err, y_type)
    bad = ~(np.abs(np64(got) - Y) <= tol)
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[0], np64(got)[bad][0], Y[bad][0], tol[bad][0])


def gemv_case(M, N, K, group, asym, x_type, s_type, y_type, wide=False):
    rng = np.random.default_rng(M + N + K)
    (q, s, z), dev = make_weights(rng, (N,), K, group, asym, s_type, wide)
    x, X = make_x(rng, (M, K), x_type)
    guard = torch.full((M + 2, N), -777.0, dtype=TYPES[y_type], device="cuda")
    pad = (-N * guard.element_size()) % 16                # the second row of the guard need not be aligned
    Y = guard[1:-1] if pad == 0 else torch.empty((M, N), dtype=TYPES[y_type], device="cuda")
    got, algo = ssn.gemv_int4(X, *dev, group=group, Y=Y)
    assert got is Y and algo == ssn.ALGO_MFMA
    want, B = int4.product(x, q, s, z, group)
    check_product(got, want, int4.product_error(B, K, group), y_type)
    assert bool((guard[0] == -777).all()) and bool((guard[-1] == -777).all())
    again = ssn.gemv_int4(X, *dev, group=group, y_dtype=TYPES[y_type])[0]
    assert torch.equal(got, again)                        # one order of additions, whatever runs beside it


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 130])
def test_gemv_rows(M):
    gemv_case(M, 160, 1024, 128, True, "bf16", "bf16", "f32")


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 32, 33, 63, 65, 255, 1000, 4097])
def test_gemv_columns(N):
    gemv_case(3, N, 512, 64, True, "f16", "f16", "f16")
    gemv_case(20, N, 160, 128, False, "bf16", "f16", "f32")


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (128, 128), (160, 64), (256, 256), (512, 64),
                                     (1056, 96), (2080, 64), (2080, 128), (5120, 128), (5120, 5120), (5152, 64),
                                     (5152, 160), (8192, 1024), (96, 4096), (4128, 4128), (16384, 32)])
@pytest.mark.parametrize("M", [1, 7, 40])
def test_gemv_lengths_and_groups(M, K, group):
    gemv_case(M, 48, K, group, True, "bf16", "bf16", "f32")


@pytest.mark.parametrize("x_type,s_type,y_type", [(x, s, y) for x in ("bf16", "f16") for s in ("bf16", "f16")
                                                  for y in ("f32", "bf16", "f16")])
@pytest.mark.parametrize("asym", [False, True])
def test_gemv_types(x_type, s_type, y_type, asym):
    gemv_case(1, 64, 288, 96, asym, x_type, s_type, y_type, wide=True)
    gemv_case(18, 64, 256, 128, asym, x_type, s_type, y_type, wide=True)


@pytest.mark.parametrize("M,K,group", [(1, 160, 32), (16, 160, 128), (40, 160, 64), (64, 256, 256)])
@pytest.mark.parametrize("x_type", ["bf16", "f16"])
def test_gemv_of_unit_vectors_gives_the_weights(M, K, group, x_type):
    """x = e_k: s (q - z) is exact in f32, whatever the order; every k and n is seen."""
    rng = np.random.default_rng(K)
    N = 40
    (q, s, z), dev = make_weights(rng, (N,), K, group, True, "bf16")
    W = int4.dequantize(q, s, z, group)
    for k0 in range(0, K, M):
        X = torch.zeros((M, K), dtype=TYPES[x_type], device="cuda")
        rows = min(M, K - k0)
        X[torch.arange(rows), torch.arange(k0, k0 + rows)] = 1
        got = np64(ssn.gemv_int4(X, *dev, group=group)[0])
        assert np.array_equal(got[:rows], W[:, k0:k0 + rows].T) and not got[rows:].any()


@pytest.mark.parametrize("M", [2, 20, 64])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_gemv_non_finite_rows_stay_in_their_row(M, bad):
    rng = np.random.default_rng(M)
    (q, s, z), dev = make_weights(rng, (96,), 512, 128, True, "bf16")
    x, X = make_x(rng, (M, 512), "bf16")
    clean = ssn.gemv_int4(X, *dev)[0].clone()
    X[1, 300] = bad
    got = ssn.gemv_int4(X, *dev)[0]
    assert not bool(torch.isfinite(got[1]).any())
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("M", [1, 12, 40])
def test_gemv_keeps_subnormal_halves(M):
    """Activations below f16's smallest normal number, 2^-14, count as they are."""
    rng = np.random.default_rng(M)
    (q, s, z), dev = make_weights(rng, (40,), 512, 128, True, "f16")
    X = torch.from_numpy(rng.integers(-1000, 1001, (M, 512)) * 2.0 ** -24).half()
    want, B = int4.product(np64(X), q, s, z, 128)
    check_product(ssn.gemv_int4(X.cuda(), *dev)[0], want, int4.product_error(B, 512, 128), "f32")


def test_gemv_unaligned_scales_and_zeros():
    """Scales and zero points of one part of a larger array: 2-byte and 1-byte aligned."""
    rng = np.random.default_rng(8)
    (q, s, z), (codes, scales, zeros) = make_weights(rng, (33,), 224, 96, True, "f16")
    x, X = make_x(rng, (2, 224), "f16")
    s2 = torch.zeros(1 + scales.numel(), dtype=scales.dtype, device="cuda")[1:].view_as(scales).copy_(scales)
    z2 = torch.zeros(3 + zeros.numel(), dtype=zeros.dtype, device="cuda")[3:].view_as(zeros).copy_(zeros)
    assert s2.data_ptr() % 4 == 2 and z2.data_ptr() % 2 == 1
    assert torch.equal(ssn.gemv_int4(X, codes, s2, z2, group=96)[0], ssn.gemv_int4(X, codes, scales, zeros, group=96)[0])


def test_gemv_beyond_4_gib_of_codes():
    """Rows whose codes start past 2^32 bytes."""
    K, N = 8192, (1 << 20) + 40
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((N, K // 1024), generator=g, device="cuda") * 0.01).to(torch.bfloat16)
    zeros = torch.randint(0, 16, (N, K // 1024), generator=g, device="cuda", dtype=torch.uint8)
    x, X = make_x(np.random.default_rng(0), (2, K), "bf16")
    got = ssn.gemv_int4(X, codes, scales, zeros, group=1024)[0]
    rows = torch.tensor([0, 1, (1 << 19) - 1, 1 << 19, (1 << 20) - 1, 1 << 20, N - 2, N - 1], device="cuda")
    q, s, z = int4.unpack(codes[rows].cpu().numpy()), np64(scales[rows]), zeros[rows].cpu().numpy().astype(np.int64)
    want, B = int4.product(x, q, s, z, 1024)
    check_product(got[:, rows], want, int4.product_error(B, K, 1024), "f32")


def sampled_case(M, N, K, group, asym, x_type="bf16", s_type="bf16", y_type="f32"):
    """A product too large for the oracle, checked on weight rows spread over all of it, the last among them."""
    g = torch.Generator(device="cuda").manual_seed(N + K + M)
    groups = -(-K // group)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((N, groups), generator=g, device="cuda") * 0.01).to(TYPES[s_type])
    zeros = torch.randint(0, 16, (N, groups), generator=g, device="cuda", dtype=torch.uint8) if asym else None
    x, X = make_x(np.random.default_rng(M), (M, K), x_type)
    Y = torch.full((M, N), float("nan"), dtype=TYPES[y_type], device="cuda")
    ssn.gemv_int4(X, codes, scales, zeros, group=group, Y=Y)
    assert bool(torch.isfinite(Y).all())
    rows = torch.unique(torch.cat((torch.arange(0, N, max(1, N // 40)), torch.arange(max(0, N - 20), N)))).cuda()
    q, s = int4.unpack(codes[rows].cpu().numpy()), np64(scales[rows])
    z = zeros[rows].cpu().numpy().astype(np.int64) if asym else np.full(s.shape, 8)
    want, B = int4.product(x, q, s, z, group)
    check_product(Y[:, rows], want, int4.product_error(B, K, group), y_type)


# 9 to 16 rows over many weight rows (activations in registers, one operand per row set); more waves and chunks
@pytest.mark.parametrize("M", [9, 16])
@pytest.mark.parametrize("K,group", [(96, 32), (1024, 128), (4096, 64), (4224, 128), (5152, 64), (6272, 32), (8192, 128),
                                     (8160, 96), (7200, 7200)])
def test_gemv_many_weight_rows(M, K, group):
    sampled_case(M, 16500, K, group, True, *(("f16", "bf16", "f16") if K == 4224 else ()))


# tiles of 16, 32 and 64 weight rows times one, two and four row tiles
@pytest.mark.parametrize("M", [12, 20, 64, 130])
@pytest.mark.parametrize("N", [100, 6200, 12300])
@pytest.mark.parametrize("K,group", [(160, 64), (1056, 96), (2048, 128), (2080, 128)])
def test_gemv_tile_shapes(M, N, K, group):
    sampled_case(M, N, K, group, K != 1056, "f16" if N == 6200 else "bf16")


@pytest.mark.parametrize("M,N", [(13, 1000), (13, 6150), (13, 10230), (13, 12345),      # one row tile, 1 to 4 column tiles
                                 (29, 4090), (29, 8190), (29, 10230), (29, 12345),     # two
                                 (61, 8190), (61, 10230), (61, 13801), (130, 12290)])  # four, 2 to 4 column tiles
@pytest.mark.parametrize("K,group,x_type", [(1184, 32, "f16"), (1184, 64, "bf16"), (1056, 128, "bf16")])
def test_gemv_row_and_column_tiles(M, N, K, group, x_type):
    sampled_case(M, N, K, group, True, x_type)


@pytest.mark.parametrize("M", [1, 4, 5, 16])
@pytest.mark.parametrize("K,group", [(8224, 32), (12320, 128), (16352, 64), (16384, 16384), (16416, 96), (40000, 128)])
def test_gemv_long_rows(M, K, group):
    sampled_case(M, 70, K, group, True)


def test_gemv_at_the_longest_row():
    sampled_case(2, 3, 1 << 20, 128, True)


def test_two_products_at_once():
    """Two streams, other inputs: nothing is shared between calls."""
    rng = np.random.default_rng(12)
    sets = []
    for i in range(2):
        _, dev = make_weights(rng, (2048,), 1024, 128, True, "bf16")
        sets.append((make_x(rng, (6 + 12 * i, 1024), "bf16")[1], dev, torch.cuda.Stream()))
    want = [ssn.gemv_int4(X, *dev)[0] for X, dev, _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (X, dev, stream) in enumerate(sets):
            with torch.cuda.stream(stream):
                got[i].append(ssn.gemv_int4(X, *dev)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


# ------------------------------------------------------------------------------ grouped product
def grouped_case(counts, R, x_rows, N, K, group, asym, silu, x_type="bf16", s_type="bf16", y_type="f32", gather=True):
    """counts: rows of each expert; R >= their sum (rows behind them belong to no expert)."""
    E = len(counts)
    rng = np.random.default_rng(N + K + R)
    (q, s, z), dev = make_weights(rng, (E, N), K, group, asym, s_type)
    x, X = make_x(rng, (x_rows, K), x_type)
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    src = rng.integers(0, x_rows, R).astype(np.int32) if gather else np.arange(R)
    No = N // 2 if silu else N
    Y = torch.full((R, No), -777.0, dtype=TYPES[y_type], device="cuda")
    got, algo = ssn.moe_grouped_gemv_int4(X, torch.from_numpy(src).cuda() if gather else None,
                                          torch.from_numpy(off).cuda(), R, *dev, group=group,
                                          epilogue=ssn.EPI_SILU_GATE if silu else ssn.EPI_NONE, Y=Y)
    assert got is Y and algo == ssn.ALGO_STREAM
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        want, B = int4.product(x[src[a:b]], q[e], s[e], z[e], group)
        err = int4.product_error(B, K, group)
        if silu:
            want, err = int4.silu_gate(want[:, :No], want[:, No:], err[:, :No], err[:, No:])
        check_product(got[a:b], want, err, y_type)
    assert bool((got[off[-1]:] == -777).all())            # rows of no expert


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts,extra", [([1], 0), ([0, 3, 0, 0, 5, 1, 0], 0), ([16, 17, 33, 1, 0, 64], 3),
                                          ([0, 0, 0], 2), ([200], 0), ([1] * 70, 1)])
def test_grouped_counts(counts, extra, silu):
    grouped_case(counts, sum(counts) + extra, 9, 96, 256, 128, True, silu)


@pytest.mark.parametrize("N", [2, 30, 32, 34, 66, 130])
@pytest.mark.parametrize("silu", [False, True])
def test_grouped_columns(N, silu):
    grouped_case([2, 0, 19, 1], 22, 5, N, 160, 64, False, silu, "f16", "f16", "f16")


@pytest.mark.parametrize("K,group", [(32, 32), (512, 64), (2048, 128), (2080, 96), (512, 512), (4096, 32)])
@pytest.mark.parametrize("silu", [False, True])
def test_grouped_lengths(K, group, silu):
    grouped_case([1, 2, 0, 18], 21, 21, 64, K, group, True, silu, "bf16", "f16", "bf16", gather=False)


@pytest.mark.parametrize("K,group", [(8224, 32), (12320, 96), (16416, 128), (8320, 8320)])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_long_rows(K, group, silu, gather):
    grouped_case([3, 0, 18], 22, 22, 34, K, group, True, silu, "bf16", "f16", "bf16", gather=gather)
    grouped_case([1, 2], 3, 3, 34, K, group, False, silu, "f16", "f16", "f32", gather=gather)


def test_grouped_unequal_experts():
    """One expert with most rows beside many with one: sets of rows are dealt to workgroups on the device."""
    grouped_case([1] * 30 + [700] + [0] * 20 + [1] * 13, 743, 40, 64, 128, 64, True, True)


def test_grouped_many_experts():
    counts = [0] * 2048
    counts[0] = counts[1023] = counts[1024] = counts[2047] = 2
    grouped_case(counts, 8, 8, 32, 64, 64, True, False)


def test_grouped_clamps_what_it_reads():
    """Offsets beyond R and tokens outside X are taken to their nearest valid value, as documented."""
    rng = np.random.default_rng(2)
    (q, s, z), dev = make_weights(rng, (3, 32), 64, 32, True, "bf16")
    x, X = make_x(rng, (4, 64), "bf16")
    tok = torch.tensor([-5, 2, 100, 1], dtype=torch.int32, device="cuda")
    off = torch.tensor([-3, 2, 9, 1000], dtype=torch.int32, device="cuda")
    got = ssn.moe_grouped_gemv_int4(X, tok, off, 4, *dev, group=32)[0]
    for r, (e, t) in enumerate(((0, 0), (0, 2), (1, 3), (1, 1))):
        want, B = int4.product(x[t:t + 1], q[e], s[e], z[e], 32)
        check_product(got[r:r + 1], want, int4.product_error(B, 64, 32), "f32")


def test_grouped_rows_equal_the_plain_product():
    """Per expert, the grouped product adds in the plain product's order of the same rows."""
    rng = np.random.default_rng(4)
    (q, s, z), (codes, scales, zeros) = make_weights(rng, (3, 64), 512, 128, True, "bf16")
    x, X = make_x(rng, (12, 512), "bf16")
    off = torch.tensor([0, 4, 4, 12], dtype=torch.int32, device="cuda")
    got = ssn.moe_grouped_gemv_int4(X, None, off, 12, codes, scales, zeros)[0]
    for e, a, b in ((0, 0, 4), (2, 4, 12)):
        y = ssn.gemv_int4(X[a:b].contiguous(), codes[e], scales[e], zeros[e])[0]
        assert (got[a:b] - y).abs().max() <= 1e-5 * y.abs().max()


# ------------------------------------------------------------------------------ use
def test_prepared_calls_streams_and_graph_replays():
    rng = np.random.default_rng(6)
    (q, s, z), dev = make_weights(rng, (128,), 512, 128, True, "bf16")
    X = make_x(rng, (4, 512), "bf16")[1]
    W = torch.from_numpy(np.float32(rng.standard_normal((32, 256)))).cuda()
    off = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    gw = [t.view(2, 64, -1) for t in dev]

    def all_calls():
        y = ssn.gemv_int4(X, *dev)[0]
        g = ssn.moe_grouped_gemv_int4(X, None, off, 4, *gw, epilogue=ssn.EPI_SILU_GATE)[0]
        c = ssn.int4_quantize(W, group=64)
        return (y, g, *c, ssn.int4_dequantize(*c, group=64))

    call, (Y, used) = ssn.gemv_int4(X, *dev, prepare=True)
    call()
    assert used.value == ssn.ALGO_MFMA and torch.equal(Y, all_calls()[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_calls()
    for seed in (1, 2, 3):                                # new inputs in place, eager work between the replays
        r = np.random.default_rng(seed)
        X.copy_(make_x(r, (4, 512), "bf16")[1])
        W.copy_(torch.from_numpy(np.float32(r.standard_normal((32, 256)))))
        want = [t.clone() for t in all_calls()]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_misaligned_tensors_are_refused():
    X = torch.zeros((3, 32), dtype=torch.bfloat16, device="cuda").view(-1)[8:72]     # 16 bytes on: aligned
    c, s = torch.zeros((4, 16), dtype=torch.uint8, device="cuda"), torch.zeros((4, 1), dtype=torch.bfloat16, device="cuda")
    ssn.gemv_int4(X.view(2, 32), c, s, group=32)
    with pytest.raises(ssn.SsnError, match="X.*aligned"):
        ssn.gemv_int4(torch.zeros(65, dtype=torch.bfloat16, device="cuda")[1:].view(2, 32), c, s, group=32)
    with pytest.raises(ValueError, match="contiguous"):
        ssn.gemv_int4(torch.zeros((32, 2), dtype=torch.bfloat16, device="cuda").t(), c, s, group=32)


def test_tensors_on_two_devices_are_refused():
    rng = np.random.default_rng(6)
    _, (codes, scales, zeros) = make_weights(rng, (32,), 64, 32, True, "bf16")
    X = make_x(rng, (1, 64), "bf16")[1]
    with pytest.raises(ValueError, match="device"):
        ssn.gemv_int4(X, codes, scales.cpu(), zeros, group=32)
    with pytest.raises(ValueError, match="shape"):
        ssn.gemv_int4(X, codes, scales, zeros, group=64)
    with pytest.raises(ssn.SsnError):
        ssn.gemv_int4(X, codes, scales, zeros, group=32, algo=ssn.ALGO_VALU)
