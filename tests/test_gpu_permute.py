"""GPU parity of moe_permute, moe_unpermute and their gradients against the float64 oracle, and the run of a
mixture of experts with integer 4-bit weights through them."""
import numpy as np
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn
import synth
from oracle import int4, moe, permute

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def np64(t):
    return t.detach().cpu().double().numpy()


def routing(rng, T, k, R, drop):
    """row_of with T k - drop entries placed on rows of [0, R) and the others outside it."""
    F = T * k
    row_of = np.full(F, -1, np.int32)
    placed = rng.permutation(F)[:F - drop]
    row_of[placed] = rng.permutation(R)[:F - drop]
    lost = np.setdiff1d(np.arange(F), placed)
    row_of[lost[::2]] = R + rng.integers(0, 5, lost[::2].size)      # beyond the rows, as well as -1
    return row_of


def tensor(rng, shape, t):
    v = torch.from_numpy(rng.standard_normal(shape)).to(TYPES[t])
    return np64(v), v.cuda()


def check(got, want, err, t):
    tol = err + int4.rounding(np.abs(want) + err, t)
    bad = ~(np.abs(np64(got) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[0], np64(got)[bad][0], want[bad][0], tol[bad][0])


def case(T, k, D, spare, drop, weighted, x_type, out_type=None):
    """All four calls on one routing; `spare` rows that no entry owns keep what they held."""
    out_type = out_type or x_type
    rng = np.random.default_rng(T * k + D)
    R = T * k - drop + spare
    row_of = routing(rng, T, k, R, drop)
    dro = torch.from_numpy(row_of).cuda()
    w = np.float32(rng.random((T, k)) + 0.1) if weighted else None
    dw = torch.from_numpy(w).cuda() if weighted else None
    owned = torch.zeros(R, dtype=torch.bool)
    owned[torch.from_numpy(row_of[(row_of >= 0) & (row_of < R)]).long()] = True

    def scattered(got, A, t):
        want = permute.scatter(A, row_of, w, R, np.full((R, D), -777.0))
        check(got, want, int4.U32 * np.abs(want) if weighted else 0 * want, t)
        assert bool((got.cpu()[~owned] == -777).all())

    x, X = tensor(rng, (T, D), x_type)
    Xp = torch.full((R, D), -777.0, dtype=TYPES[x_type], device="cuda")
    got = ssn.moe_permute(X, dro, dw, R=R, Xp=Xp)
    assert got is Xp
    scattered(got, x, x_type)

    g, G = tensor(rng, (R, D), x_type)
    dX, dweights = ssn.moe_permute_backward(G, dro, T, dw, X=X)
    want, mag = permute.gather(g, row_of, w, T)
    check(dX, want, permute.gather_error(mag, k), x_type)
    dots, dmag = permute.dots(x, g, row_of)
    check(dweights, dots, permute.dot_error(dmag, D), "f32")
    alone, none = ssn.moe_permute_backward(G, dro, T, dw)
    assert none is None and torch.equal(alone, dX)

    y, Y = tensor(rng, (R, D), x_type)
    out = ssn.moe_unpermute(Y, dro, T, dw, out_dtype=TYPES[out_type])
    want, mag = permute.gather(y, row_of, w, T)
    check(out, want, permute.gather_error(mag, k), out_type)

    h, H = tensor(rng, (T, D), out_type)
    dYp = torch.full((R, D), -777.0, dtype=TYPES[x_type], device="cuda")
    dYp, dweights = ssn.moe_unpermute_backward(H, dro, R, dw, Yp=Y, dYp=dYp)
    scattered(dYp, h, x_type)
    dots, dmag = permute.dots(h, y, row_of)
    check(dweights, dots, permute.dot_error(dmag, D), "f32")
    spare_rows = torch.full((R, D), -777.0, dtype=TYPES[x_type], device="cuda")
    alone, none = ssn.moe_unpermute_backward(H, dro, R, dw, y_dtype=TYPES[x_type], dYp=spare_rows)
    assert none is None and torch.equal(alone, dYp)


@pytest.mark.parametrize("x_type,out_type", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                             ("f16", "f32")])
@pytest.mark.parametrize("weighted", [False, True])
def test_types(x_type, out_type, weighted):
    case(37, 4, 264, 3, 11, weighted, x_type, out_type)
    case(5, 3, 99, 0, 2, weighted, x_type, out_type)


@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 512, 1001, 2047, 2048, 2049, 4100, 10007])
def test_widths(D):
    case(6, 3, D, 2, 1, True, "bf16")
    case(3, 2, D, 0, 0, True, "f32")


@pytest.mark.parametrize("T,k", [(1, 1), (1, 10), (2, 64), (63, 9), (300, 8), (1030, 6), (17, 33)])
def test_tokens_and_slots(T, k):
    case(T, k, 72, 0, 0, True, "f16")
    case(T, k, 40, 1, min(T * k - 1, 5), True, "f32", "f32")


def test_no_entry_has_a_row():
    T, k, D = 3, 2, 40
    dro = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    Y = torch.full((4, D), float("nan"), device="cuda")
    w = torch.ones((T, k), device="cuda")
    assert not bool(ssn.moe_unpermute(Y, dro, T, w).any())
    dX, dw = ssn.moe_permute_backward(Y, dro, T, w, X=torch.full((T, D), float("inf"), device="cuda"))
    assert not bool(dX.any()) and not bool(dw.any())
    dYp, dw = ssn.moe_unpermute_backward(Y[:T], dro, 4, w, Yp=Y, dYp=torch.full((4, D), 5.0, device="cuda"))
    assert bool((dYp == 5).all()) and not bool(dw.any())
    # no rows at all
    E = torch.empty((0, D), device="cuda")
    assert not bool(ssn.moe_unpermute(E, dro, T, w).any())
    dYp, dw = ssn.moe_unpermute_backward(Y[:T], dro, 0, w, Yp=E)
    assert dYp.shape == (0, D) and not bool(dw.any())


def test_empty():
    dro = torch.zeros(0, dtype=torch.int32, device="cuda")
    X = torch.empty((0, 16), device="cuda")
    assert ssn.moe_permute(X, dro).shape == (0, 16) and ssn.moe_unpermute(X, dro, 0).shape == (0, 16)
    Z = torch.empty((3, 0), device="cuda")                       # no columns: the weights' gradients are 0
    dro = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    w = torch.ones((3, 1), device="cuda")
    out = torch.full((3, 1), 7.0, device="cuda")
    assert not bool(ssn.moe_permute_backward(Z, dro, 3, w, X=Z, dweights=out)[1].any())
    out.fill_(7.0)
    assert not bool(ssn.moe_unpermute_backward(Z, dro, 3, w, Yp=Z, dweights=out)[1].any())


def test_non_finite_values_reach_only_their_rows():
    rng = np.random.default_rng(1)
    dro = torch.tensor([3, 0, 1, 2], dtype=torch.int32, device="cuda")
    _, Y = tensor(rng, (4, 24), "bf16")
    w = torch.tensor([[0.5, 0.0], [1.0, 2.0]], device="cuda")
    clean = ssn.moe_unpermute(Y, dro, 2, w)
    Y[0, 5] = float("inf")                                       # slot 1 of token 0, whose weight is 0
    got = ssn.moe_unpermute(Y, dro, 2, w)
    assert bool(torch.isnan(got[0, 5])) and torch.equal(got[1], clean[1])
    keep = torch.arange(24, device="cuda") != 5
    assert torch.equal(got[0][keep], clean[0][keep])


def test_weights_of_entries_without_a_row_are_not_read():
    dro = torch.tensor([1, -1, 0, 7], dtype=torch.int32, device="cuda")          # two entries without a row
    w = torch.tensor([[0.5, float("nan")], [2.0, float("inf")]], device="cuda")
    Y = torch.ones((2, 10), device="cuda")
    assert torch.equal(ssn.moe_unpermute(Y, dro, 2, w), torch.tensor([[0.5], [2.0]], device="cuda").expand(2, 10))
    dX, dw = ssn.moe_permute_backward(Y, dro, 2, w, X=Y)
    assert torch.equal(dw, torch.tensor([[10.0, 0.0], [10.0, 0.0]], device="cuda")) and bool(torch.isfinite(dX).all())
    assert torch.equal(ssn.moe_permute(Y, dro, w, R=2)[:, 0], torch.tensor([2.0, 0.5], device="cuda"))


def test_two_calls_at_once():
    rng = np.random.default_rng(10)
    T, k, D = 300, 6, 520
    sets = [(torch.from_numpy(routing(rng, T, k, T * k, 0)).cuda(), torch.rand((T, k), device="cuda"),
             tensor(rng, (T, D), "bf16")[1], tensor(rng, (T * k, D), "bf16")[1], torch.cuda.Stream()) for _ in range(2)]

    def both(ro, w, X, Y):
        return (*ssn.moe_permute_backward(Y, ro, T, w, X=X), *ssn.moe_unpermute_backward(X, ro, T * k, w, Yp=Y))
    want = [both(*s[:4]) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(sets):
            with torch.cuda.stream(s[4]):
                got[i].append(both(*s[:4]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


def test_unweighted_permutation_is_a_copy_bit_for_bit():
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).cuda()     # every 16-bit pattern, NaNs among them
    for t in (torch.bfloat16, torch.float16):
        X = bits.view(256, 256).view(t)
        dro = torch.from_numpy(np.random.default_rng(0).permutation(512).astype(np.int32)).cuda()
        Xp = ssn.moe_permute(X, dro)
        assert torch.equal(Xp.view(torch.int16)[dro.long()], X.view(torch.int16).repeat_interleave(2, 0))


def test_the_combine_is_the_weighted_f32_case():
    rng = np.random.default_rng(3)
    ids, w = synth.routing(50, 64, 6, 1.1, seed=2)
    off, rt, rs, ro, bad = ssn.moe_route(torch.from_numpy(ids).cuda(), 64)
    W = torch.from_numpy(w).cuda()
    for t in ("f32", "bf16"):
        Y = tensor(rng, (300, 200), t)[1]
        assert torch.equal(ssn.moe_combine(Y, ro, W), ssn.moe_unpermute(Y, ro, 50, W, out_dtype=torch.float32))


def test_rows_beyond_2_gib():
    """Row offsets past 2^31 and 2^32 bytes."""
    D, R = 4096 * 256, 2400                                      # 5 GB of rows
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn((3, D), generator=g, device="cuda").to(torch.bfloat16)
    dro = torch.tensor([2399, 1100, 2, 2100, -1, 1024], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0], [4.0, 0.5], [8.0, 0.25]], device="cuda")   # products without rounding
    Xp = ssn.moe_permute(X, dro, w, R=R)
    for f, r in enumerate(dro.tolist()):
        if r >= 0:
            assert torch.equal(Xp[r], X[f // 2] * w.view(-1)[f].to(torch.bfloat16))
    out = ssn.moe_unpermute(Xp, dro, 3, out_dtype=torch.float32)
    assert torch.equal(out[0], Xp[2399].float() + Xp[1100].float())
    assert torch.equal(out[1], Xp[2].float() + Xp[2100].float())
    assert torch.equal(out[2], Xp[1024].float())


@pytest.mark.parametrize("T,k,D,t,dout_t", [(2100, 16, 2001, "f32", "f32"), (7000, 16, 601, "f32", "f32"),
                                            (14000, 16, 301, "f32", "f32"), (4200, 16, 2001, "bf16", "bf16"),
                                            (4200, 16, 2001, "f16", "f32"), (28000, 16, 303, "bf16", "f32")])
def test_rows_beyond_the_cache(T, k, D, t, dout_t):
    """Rows of 268 MB and more, which are written past the caches."""
    g = torch.Generator(device="cuda").manual_seed(D)
    X = torch.randn((T, D), generator=g, device="cuda").to(TYPES[t])
    row_of = torch.randperm(T * k, generator=g, device="cuda").int()
    row_of[5] = -1
    owned = row_of.long().clamp(min=0)
    keep = row_of >= 0
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    Xp = torch.zeros((T * k, D), dtype=TYPES[t], device="cuda")
    ssn.moe_permute(X, row_of, Xp=Xp)
    assert torch.equal(Xp[owned[keep]], X.repeat_interleave(k, 0)[keep])
    dout = torch.randn((T, D), generator=g, device="cuda").to(TYPES[dout_t])
    dYp, dw = ssn.moe_unpermute_backward(dout, row_of, T * k, w, Yp=Xp)
    # one product, rounded to the type: to f32 first (half a step 2^-24) or, with halves, in one instruction without
    half, least = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}[t]
    for j in range(k):
        mine = keep.view(T, k)[:, j]
        want = (w[:, j:j + 1].double() * dout.double())[mine]
        off = (dYp[owned.view(T, k)[:, j]][mine].double() - want).abs()
        assert bool((off <= (half * (1 + 2.0 ** -24) + 2.0 ** -24) * want.abs() + least).all())
    a, b = dout.double(), X.double()
    err = (D + 16) * 2.0 ** -24 * (a * b).abs().sum(1, keepdim=True)
    assert bool(((dw - (a * b).sum(1, keepdim=True)).abs() <= err)[keep.view(T, k)].all()) and dw[0, 5] == 0


# T k D elements of 268 MB and more; a wave, two or four to a token, rows of fewer elements than a lane moves, whole
# vectors and a last one that overlaps
@pytest.mark.parametrize("T,k,D,t,dout_t", [
    (14000, 16, 301, "f32", "f32"), (7000, 16, 601, "f32", "f32"), (2100, 16, 2001, "f32", "f32"), (210000, 64, 5, "f32", "f32"),
    (28000, 16, 303, "bf16", "bf16"), (14000, 16, 601, "bf16", "bf16"), (4100, 16, 2048, "bf16", "bf16"),
    (28000, 16, 303, "f16", "f16"), (14000, 16, 601, "f16", "f16"), (4200, 16, 2001, "f16", "f16"),
    (28000, 16, 303, "bf16", "f32"), (14000, 16, 601, "bf16", "f32"), (4200, 16, 2001, "bf16", "f32"),
    (28000, 16, 303, "f16", "f32"), (14000, 16, 601, "f16", "f32"), (4100, 16, 2048, "f16", "f32")])
def test_weighted_rows_beyond_the_cache(T, k, D, t, dout_t):
    """The weighted movements that write such rows past the caches: moe_unpermute_backward without dweights, equal
    bit for bit to the call with dweights, which writes through them, and moe_permute with weights."""
    g = torch.Generator(device="cuda").manual_seed(T + D)
    row_of = torch.randperm(T * k, generator=g, device="cuda").int()
    lost = int(row_of[5])
    row_of[5] = -1
    keep = row_of.view(T, k) >= 0
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    # one product, rounded to the type: to f32 first (half a step 2^-24) or, with halves, in one instruction without
    half, least = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}[t]

    def scattered(rows, A):
        assert bool((rows[lost] == -777).all())
        for j in range(k):
            want = (w[:, j:j + 1].double() * A.double())[keep[:, j]]
            off = (rows[row_of.view(T, k)[:, j][keep[:, j]].long()].double() - want).abs()
            assert bool((off <= (half * (1 + 2.0 ** -24) + 2.0 ** -24) * want.abs() + least).all())

    dout = torch.randn((T, D), generator=g, device="cuda").to(TYPES[dout_t])
    dYp = torch.full((T * k, D), -777.0, dtype=TYPES[t], device="cuda")
    assert ssn.moe_unpermute_backward(dout, row_of, T * k, w, y_dtype=TYPES[t], dYp=dYp)[1] is None
    scattered(dYp, dout)
    with_dw = torch.full((T * k, D), -777.0, dtype=TYPES[t], device="cuda")
    ssn.moe_unpermute_backward(dout, row_of, T * k, w, Yp=dYp, dYp=with_dw)
    assert torch.equal(with_dw, dYp)
    del with_dw
    if t == dout_t:
        dYp.fill_(-777.0)
        ssn.moe_permute(dout, row_of, w, R=T * k, Xp=dYp)
        scattered(dYp, dout)


def test_graph_replays():
    rng = np.random.default_rng(9)
    T, k, D = 40, 5, 136
    row_of = routing(rng, T, k, T * k, 0)
    dro, w = torch.from_numpy(row_of).cuda(), torch.rand((T, k), device="cuda")
    X, G = tensor(rng, (T, D), "bf16")[1], tensor(rng, (T * k, D), "bf16")[1]

    def all_calls():
        return (ssn.moe_permute(X, dro, w), *ssn.moe_permute_backward(G, dro, T, w, X=X), ssn.moe_unpermute(G, dro, T, w),
                *ssn.moe_unpermute_backward(X, dro, T * k, w, Yp=G))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_calls()
    for seed in (1, 2, 3):
        X.copy_(tensor(np.random.default_rng(seed), (T, D), "bf16")[1])
        G.copy_(tensor(np.random.default_rng(seed + 9), (T * k, D), "bf16")[1])
        dro.copy_(torch.from_numpy(routing(np.random.default_rng(seed), T, k, T * k, 0)))
        want = [t.clone() for t in all_calls()]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------ a run of the operators together
@pytest.mark.parametrize("T", [1, 7, 60])
def test_mixture_of_experts_with_int4_weights(T):
    """Route, tokens to expert order, gate and up, down, back with the routing weights; then the gradient of the
    weighted sum. Against the oracle on the quantised weights, stage by stage on the GPU's own intermediates."""
    E, k, D, I, group = 24, 4, 256, 96, 32
    rng = np.random.default_rng(T)
    ids, w = synth.routing(T, E, k, 1.1, seed=T)
    x_bits = synth.activations(T, D, seed=T)
    X = torch.from_numpy(x_bits.view(np.int16)).view(torch.bfloat16).cuda()
    up = ssn.int4_quantize(torch.from_numpy(np.concatenate([synth.expert_up(e, I, D) for e in range(E)])).cuda(), group)
    down = ssn.int4_quantize(torch.from_numpy(np.concatenate([synth.expert_down(e, I, D) for e in range(E)])).cuda(), group)
    up, down = [t.view(E, 2 * I, -1) for t in up], [t.view(E, D, -1) for t in down]
    W = torch.from_numpy(w).cuda()

    off, row_token, _, row_of, bad = ssn.moe_route(torch.from_numpy(ids).cuda(), E)
    Xp = ssn.moe_permute(X, row_of)
    H, _ = ssn.moe_grouped_gemv_int4(Xp, None, off, T * k, *up, group=group, epilogue=ssn.EPI_SILU_GATE,
                                     y_dtype=torch.bfloat16)
    H2, _ = ssn.moe_grouped_gemv_int4(X, row_token, off, T * k, *up, group=group, epilogue=ssn.EPI_SILU_GATE,
                                      y_dtype=torch.bfloat16)
    Yp, _ = ssn.moe_grouped_gemv_int4(H, None, off, T * k, *down, group=group, y_dtype=torch.bfloat16)
    out = ssn.moe_unpermute(Yp, row_of, T, W)
    dout = torch.from_numpy(rng.standard_normal((T, D))).to(torch.bfloat16).cuda()
    dYp, dweights = ssn.moe_unpermute_backward(dout, row_of, T * k, W, Yp=Yp)
    torch.cuda.synchronize()
    assert int(bad.item()) == 0
    assert torch.equal(H, H2)                                    # gathered inside the product, or before it

    _, offsets, rt, _ = moe.route(ids, E)
    ro = row_of.cpu().numpy()
    assert np.array_equal(np64(Xp), np64(X)[rt])

    def parts(t):
        codes, s, z = t
        return int4.unpack(codes.cpu().numpy()), np64(s), z.cpu().numpy().astype(np.int64)
    (uq, us, uz), (dq, ds, dz) = parts(up), parts(down)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        gu, B = int4.product(np64(Xp)[a:b], uq[e], us[e], uz[e], group)
        err = int4.product_error(B, D, group)
        h, eh = int4.silu_gate(gu[:, :I], gu[:, I:], err[:, :I], err[:, I:])
        check(H[a:b], h, eh, "bf16")
        y, B = int4.product(np64(H)[a:b], dq[e], ds[e], dz[e], group)
        check(Yp[a:b], y, int4.product_error(B, I, group), "bf16")
    o, mag = permute.gather(np64(Yp), ro, w, T)
    check(out, o, permute.gather_error(mag, k), "bf16")
    d = permute.scatter(np64(dout), ro, w, T * k, np.zeros((T * k, D)))
    check(dYp, d, int4.U32 * np.abs(d), "bf16")
    dots, dmag = permute.dots(np64(dout), np64(Yp), ro)
    check(dweights, dots, permute.dot_error(dmag, D), "f32")
