"""GPU parity of the 4-bit cache of keys and values: append and read against the float64 oracle, bit for bit."""
import numpy as np
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn
from oracle import kv

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make_cache(pages, page, H, D, ts, fill=0xAA):
    c = ssn.kv_nvfp4_empty(pages, page, D, torch.tensor(ts[0], dtype=torch.float32).cuda(),
                           torch.tensor(ts[1], dtype=torch.float32).cuda())
    for t in c[:4]:
        t.fill_(fill)
    return c


def host(cache):
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in cache[:4]]


def special_tokens(rng, T, H, D, ts):
    """Normal values with zero blocks, ties, tiny and saturating ones."""
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    if T >= 8:
        x[0] = 0.0
        x[1] = (np.arange(D) % 25 - 12).astype(np.float32) * 0.25            # ties of E2M1 for a scale of 1
        x[2] = -np.abs(x[2]) * 1e-12                                         # scales that round to 0
        x[3] *= 1e4                                                          # beyond 2688 s_h
        x[4, :, ::2] = -0.0
        x[5] *= 2.0 ** -9                                                    # subnormal scales
        x[6, :, : D - 1] = 0.0                                               # one value alone
        x[7] = np.float32(ts) * 6.0                                          # scale 1, code 6
    return x


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 32, 16), (9, 2, 64, 16), (37, 3, 96, 48), (130, 8, 128, 32),
                                        (33, 1, 160, 16), (65, 2, 224, 80), (257, 2, 256, 64), (1000, 5, 128, 256)])
def test_append_is_exact(T, H, D, page, x_type):
    rng = np.random.default_rng(T * D)
    pages = -(-T // page) + 2
    ts = (rng.random((2, H)) * 2e-3 + 5e-4).astype(np.float32)
    ts[0, 0] = 1.0
    x = [torch.from_numpy(special_tokens(rng, T, H, D, float(ts[i, 0]))).clamp(-6e4, 6e4).to(TYPES[x_type]) for i in range(2)]
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    drop = rng.random(T) < 0.1
    slots[drop] = rng.choice([-1, -7, pages * page, pages * page + 12345, 1 << 60, -(1 << 62)], int(drop.sum()))
    cache = make_cache(pages, page, H, D, ts)
    bad = torch.full((1,), 99, dtype=torch.int64, device="cuda")
    assert ssn.kv_nvfp4_append(x[0].cuda(), x[1].cuda(), torch.from_numpy(slots).cuda(), cache, bad_slots=bad) is cache
    got = host(cache)
    want = [np.full(g.shape, 0xAA, np.uint8) for g in got]
    ok = (slots >= 0) & (slots < pages * page)
    p, o = slots[ok] // page, slots[ok] % page
    for i in range(2):
        codes, scales = kv.quantize_tokens(x[i].float().numpy()[ok], ts[i])
        want[2 * i][p, :, o] = codes
        if i:
            want[3][p, :, :, o] = scales
        else:
            want[1][p, :, o] = scales
    for g, w, name in zip(got, want, ("k_codes", "k_scales", "v_codes", "v_scales")):
        assert np.array_equal(g, w), name
    assert int(bad.item()) == int((slots >= pages * page).sum())


def test_append_is_the_quantiser_of_weights():
    torch.manual_seed(0)
    T, H, D, page = 48, 2, 128, 16
    K, V = torch.randn(T, H, D, device="cuda"), torch.randn(T, H, D, device="cuda").mul_(3)
    ts = torch.tensor([[1e-3, 2e-3], [3e-3, 1e-3]], device="cuda")
    cache = ssn.kv_nvfp4_empty(3, page, D, ts[0], ts[1])
    ssn.kv_nvfp4_append(K, V, torch.arange(T, device="cuda"), cache)
    for h in range(H):
        codes, scales, _ = ssn.nvfp4_quantize(K[:, h].contiguous(), tensor_scale_in=ts[0, h:h + 1].contiguous())
        assert torch.equal(cache.k_codes[:, h].reshape(T, D // 2), codes)
        assert torch.equal(cache.k_scales[:, h].reshape(T, D // 16), scales)
        codes, scales, _ = ssn.nvfp4_quantize(V[:, h].contiguous(), tensor_scale_in=ts[1, h:h + 1].contiguous())
        assert torch.equal(cache.v_codes[:, h].reshape(T, D // 2), codes)
        assert torch.equal(cache.v_scales[:, h].transpose(1, 2).reshape(T, D // 16), scales)


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
def test_append_decides_as_the_quantiser_everywhere(x_type):
    """Three million values of every size against nvfp4_quantize (exact by its own tests): quotients next to the middle
    of two codes or scales, scales that are powers of two, tiny and huge ones, values to the end of f32."""
    g = torch.Generator(device="cuda").manual_seed(7)
    T, D, page = 2048, 256, 64
    scales = [1e-3, 2.0 ** -9, 1.0, 0.3, 1.1754944e-38, 1e-42, 1e-31, 3e38, 7e29, 2.0 ** -126, 6e-5]
    H = len(scales)
    ts = torch.tensor(scales, device="cuda")
    x = torch.randn((T, H, D), generator=g, device="cuda") * (ts[:, None] * 6).clamp(max=1e30)
    x *= torch.exp2(torch.randint(-14, 12, (T, H, D // 16, 1), generator=g, device="cuda").float()).expand(T, H, D // 16, 16).reshape(T, H, D)
    # an eighth of the blocks: multiples of s_h / 8, that is ties and their neighbours in f32
    n = torch.randint(-4000, 4000, (T // 8, H, D), generator=g, device="cuda").float()
    tie = n * (ts[:, None] / 8)
    x[: T // 8] = torch.where(torch.rand(tie.shape, generator=g, device="cuda") < 0.5, tie, torch.nextafter(tie, torch.zeros_like(tie)))
    x = x.clamp(-3e38, 3e38).nan_to_num().to(TYPES[x_type])
    if x_type == "f16":
        x = x.clamp(-65504, 65504)
    cache = ssn.kv_nvfp4_empty(T // page, page, D, ts, ts)
    ssn.kv_nvfp4_append(x, -x, torch.arange(T, device="cuda"), cache)
    for h in range(H):
        for X, codes, S in ((x, cache.k_codes, cache.k_scales), (-x, cache.v_codes, cache.v_scales.transpose(2, 3))):
            c, s, _ = ssn.nvfp4_quantize(X[:, h].float().contiguous(), tensor_scale_in=ts[h:h + 1].contiguous())
            assert torch.equal(S[:, h].reshape(T, D // 16), s), scales[h]
            assert torch.equal(codes[:, h].reshape(T, D // 2), c), scales[h]


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
def test_parts_of_one_projection(x_type):
    """K and V as slices of [T, (Hq + 2 Hkv) D], an expanded head, and a token stride of two tokens."""
    torch.manual_seed(1)
    T, Hq, H, D = 21, 4, 2, 96
    qkv = torch.randn(2 * T, Hq + 2 * H, D, device="cuda").to(TYPES[x_type])
    ts = torch.full((H,), 2e-3, device="cuda")
    slots = torch.randperm(32, device="cuda")[:T]
    for K, V in ((qkv[:T, Hq:Hq + H], qkv[:T, Hq + H:]), (qkv[::2, :H], qkv[1::2, H:2 * H]),
                 (qkv[:T, :1].expand(T, H, D), qkv[:1, :H].expand(T, H, D))):
        a, b = (ssn.kv_nvfp4_empty(2, 16, D, ts, ts) for _ in range(2))
        for t in (*a[:4], *b[:4]):
            t.zero_()
        ssn.kv_nvfp4_append(K, V, slots, a)
        ssn.kv_nvfp4_append(K.contiguous(), V.contiguous(), slots, b)
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and int(a.k_codes.count_nonzero()) > 0


def test_values_that_are_not_finite_and_scales_of_zero():
    H, D = 3, 64
    x = torch.randn(4, H, D, device="cuda")
    x[0, 0, 3], x[1, 0, 5], x[1, 0, 6] = float("nan"), float("inf"), float("-inf")
    ts = torch.tensor([1e-3, 0.0, -1.0], device="cuda")
    cache = ssn.kv_nvfp4_empty(1, 16, D, ts, ts)
    slots = torch.arange(4, device="cuda")
    ssn.kv_nvfp4_append(x, x, slots, cache)
    K, V = ssn.kv_nvfp4_read(slots, cache, out_dtype=torch.float32)
    assert torch.equal(K, V) and bool(K.isfinite().all())
    assert float(K[0, 0, 3]) == 0.0 and float(K[0, 0].abs().max()) > 0
    top = 6 * 448 * float(ts[0])
    assert abs(float(K[1, 0, 5]) - top) < 1e-6 and abs(float(K[1, 0, 6]) + top) < 1e-6
    assert int(K[:, 1:].count_nonzero()) == 0


@pytest.mark.parametrize("y_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 32, 16), (7, 2, 64, 16), (129, 3, 96, 48), (200, 8, 128, 32),
                                        (33, 1, 160, 16), (31, 2, 224, 80), (100, 2, 256, 64)])
def test_read_is_exact(T, H, D, page, y_type):
    rng = np.random.default_rng(T + D)
    pages = 5
    ts = (rng.random((2, H)) * 2e-3 + 5e-4).astype(np.float32)
    cache = make_cache(pages, page, H, D, ts)
    for t in cache[:4]:                                         # any code; any scale but NaN
        t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape).astype(np.uint8)))
    for t in (cache.k_scales, cache.v_scales):
        t.clamp_(max=0x7E)
    slots = rng.integers(0, pages * page, T)                    # the same slot more than once
    slots[rng.random(T) < 0.1] = -1
    slots[-1:] = pages * page if T > 1 else slots[-1:]
    K, V = ssn.kv_nvfp4_read(torch.from_numpy(slots).cuda(), cache, out_dtype=TYPES[y_type])
    h = host(cache)
    ok = (slots >= 0) & (slots < pages * page)
    kc, ks, vc, vs = kv.gather(*h, np.where(ok, slots, 0), page)
    for got, codes, scales, t in ((K, kc, ks, ts[0]), (V, vc, vs, ts[1])):
        # the code times the scale is exact, the product with s_h rounded to f32, then to the type asked for
        w = torch.from_numpy(np.where(ok[:, None, None], kv.dequantize_tokens(codes, scales, t), 0.0).astype(np.float32))
        assert torch.equal(got.cpu(), w.to(TYPES[y_type]))


def test_round_trip_is_the_identity():
    """What was read back is written as it was."""
    torch.manual_seed(2)
    T, H, D, page = 100, 4, 128, 16
    x = torch.randn(T, H, D, device="cuda")
    ts = torch.full((H,), 2.0 ** -9, device="cuda")
    a, b = (ssn.kv_nvfp4_empty(8, page, D, ts, ts) for _ in range(2))
    for t in (*a[:4], *b[:4]):
        t.zero_()
    slots = torch.randperm(8 * page, device="cuda")[:T]
    ssn.kv_nvfp4_append(x, -x, slots, a)
    K, V = ssn.kv_nvfp4_read(slots, a, out_dtype=torch.float32)
    ssn.kv_nvfp4_append(K, V, slots, b)
    K2, V2 = ssn.kv_nvfp4_read(slots, b, out_dtype=torch.float32)
    assert torch.equal(K, K2) and torch.equal(V, V2)


def test_no_tokens():
    ts = torch.ones(2, device="cuda")
    cache = ssn.kv_nvfp4_empty(1, 16, 64, ts, ts)
    none, bad = torch.empty(0, dtype=torch.int64, device="cuda"), torch.full((1,), 5, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 2, 64, device="cuda")
    ssn.kv_nvfp4_append(x, x, none, cache, bad_slots=bad)
    K, V = ssn.kv_nvfp4_read(none, cache)
    assert K.shape == V.shape == (0, 2, 64) and int(bad.item()) == 0


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes a tensor: its last pages."""
    H, D, page = 8, 256, 256
    pages = (1 << 32) // (H * page * D // 2) + 40
    ts = torch.full((H,), 1e-3, device="cuda")
    cache = ssn.kv_nvfp4_empty(pages, page, D, ts, ts)
    assert cache.k_codes.numel() > 1 << 32
    for t in cache[:4]:
        t[:40].fill_(0x11)
    torch.manual_seed(3)
    x = torch.randn(50, H, D, device="cuda")
    slots = (pages - 1) * page + 200 + torch.arange(50, device="cuda")
    ssn.kv_nvfp4_append(x, -x, slots, cache)
    small = ssn.kv_nvfp4_empty(1, page, D, ts, ts)
    ssn.kv_nvfp4_append(x, -x, slots - (pages - 1) * page, small)
    K, V = ssn.kv_nvfp4_read(slots, cache, out_dtype=torch.float32)
    K1, V1 = ssn.kv_nvfp4_read(slots - (pages - 1) * page, small, out_dtype=torch.float32)
    assert torch.equal(K, K1) and torch.equal(V, V1) and int(K.count_nonzero()) > 0
    assert all(bool((t[:40] == 0x11).all()) for t in cache[:4])


def test_captured_and_replayed():
    """A captured append and read with the tokens and slots of the replay's time."""
    torch.manual_seed(4)
    T, H, D, page = 16, 2, 128, 16
    ts = torch.full((H,), 1e-3, device="cuda")
    cache = ssn.kv_nvfp4_empty(4, page, D, ts, ts)
    K, V = torch.randn(T, H, D, device="cuda"), torch.randn(T, H, D, device="cuda")
    slots, bad = torch.randperm(4 * page, device="cuda")[:T], torch.zeros(1, dtype=torch.int64, device="cuda")
    ssn.kv_nvfp4_append(K, V, slots, cache, bad_slots=bad)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssn.kv_nvfp4_append(K, V, slots, cache, bad_slots=bad)
        Kr, Vr = ssn.kv_nvfp4_read(slots, cache, out_dtype=torch.float32)
    for i in range(4):
        K.copy_(torch.randn_like(K)); V.copy_(torch.randn_like(V))
        slots.copy_(torch.randperm(4 * page, device="cuda")[:T])
        slots[i] = 4 * page + i
        g.replay()
        torch.cuda.synchronize()
        other = ssn.kv_nvfp4_empty(4, page, D, ts, ts)
        ssn.kv_nvfp4_append(K, V, slots, other)
        K1, V1 = ssn.kv_nvfp4_read(slots, other, out_dtype=torch.float32)
        assert torch.equal(Kr, K1) and torch.equal(Vr, V1) and int(bad.item()) == 1
        assert int(Kr[i].count_nonzero()) == 0
