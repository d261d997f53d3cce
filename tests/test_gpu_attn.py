"""GPU parity of attention over the 4-bit cache against the float64 oracle, within the bound of its f32 evaluation."""
import numpy as np
import pytest
import torch

import structured_sparse_nvfp4_amd as ssn
from attn_util import HALF, TYPES, Batch
from oracle import kv

pytestmark = pytest.mark.gpu

STREAM, TILE = ssn.ALGO_STREAM, ssn.ALGO_MFMA
both = pytest.mark.parametrize("algo", [STREAM, TILE], ids=["stream", "tile"])

LENS = [1, 2, 15, 16, 17, 31, 32, 33, 47, 64, 65, 127, 129, 200, 255, 256, 257]


@both
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 1), (16, 2), (40, 8), (17, 1)])
def test_single_tokens(D, Hq, H, algo):
    B = Batch(LENS, [1] * len(LENS), Hq, H, D, [16, 32, 48, 64, 128][(D // 32 + Hq) % 5])
    out, lse, used = B.call(uniform=True, with_lse=True, algo=algo)
    assert used == algo and out.dtype == torch.bfloat16
    B.check(out, lse)


@both
@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_types(x, y, D, algo):
    B = Batch([300, 77, 1], [1, 3, 1], 6, 2, D, 16, x=x)
    out, lse, _ = B.call(algo=algo, out_dtype=TYPES[y], with_lse=True)
    assert out.dtype == TYPES[y]
    B.check(out, lse, out_type=y)


@both
@pytest.mark.parametrize("window", [0, 1, 2, 16, 17, 50, 4096])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 9, 16, 33])
def test_several_tokens_and_windows(n, window, algo):
    """Up to 33 queries a sequence over one, two and four sets of 16 rows; rows that leave some keys only."""
    lens = [n, n + 1, n + 15, 40 + n, 100, 257]
    B = Batch(lens, [n] * len(lens), 10, 2, 128, 16, seed=n)
    out, lse, _ = B.call(algo=algo, uniform=True, with_lse=True, window=window)
    B.check(out, lse, window=window)


@both
@pytest.mark.parametrize("D", [64, 160, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_batch(D, causal, algo):
    B = Batch([70, 0, 1, 130, 33, 290], [70, 3, 1, 7, 33, 1], 8, 4, D, 32, seed=7)
    out, lse, _ = B.call(algo=algo, with_lse=True, causal=causal)
    B.check(out, lse, causal=causal)
    assert int(out[70:73].count_nonzero()) == 0 and bool(torch.isneginf(lse[70:73]).all())


@both
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B", [2, 13, 64, 65])
def test_batches_of_many_lengths(B, causal, algo):
    """Sequences of 0 to 400 keys and 0 to 25 queries, so that each has none to four tiles of rows."""
    rng = np.random.default_rng(B)
    lens, qs = rng.integers(0, 401, B), rng.integers(0, 26, B)
    lens[0], qs[0], qs[-1] = 0, 3, 0
    X = Batch(lens.tolist(), qs.tolist(), 16, 1, 64, 16, seed=B)
    out, lse, _ = X.call(algo=algo, causal=causal, with_lse=True)
    X.check(out, lse, causal=causal)


@pytest.mark.parametrize("B,n,window,causal", [(2, 1, 0, True), (9, 1, 0, True), (40, 1, 0, True), (64, 2, 700, True), (3, 60, 0, True),
                                               (3, 60, 900, True), (5, 7, 0, False), (65, 1, 0, True)])
def test_long_sequences_among_short_ones(B, n, window, causal):
    """Two long sequences among short and empty ones, one set of rows and several."""
    rng = np.random.default_rng([B, n])
    lens = rng.integers(0, 300, B)
    lens[B // 2], lens[-1], lens[0] = 9000, 2500, 0 if B > 2 else 1200
    qs = np.minimum(rng.integers(1, n + 1, B), 60)
    qs[B // 2] = n
    X = Batch(lens.tolist(), qs.tolist(), 8, 2, 64, 64, seed=B)
    out, lse, used = X.call(algo=ssn.ALGO_STREAM, causal=causal, window=window, with_lse=True)
    X.check(out, lse, causal=causal, window=window)


@both
def test_more_queries_than_keys(algo):
    B = Batch([3, 20], [9, 20], 4, 1, 128, 16)
    out, lse, _ = B.call(algo=algo, with_lse=True)
    B.check(out, lse)
    assert int(out[:6].count_nonzero()) == 0 and bool(torch.isneginf(lse[:6]).all())


@both
def test_rows_of_no_sequence_are_left(algo):
    B = Batch([50, 60], [4, 2], 4, 2, 64, 16)
    Q = torch.cat([B.Q[:1], B.Q, B.Q[:3]])
    B.offsets = B.offsets + 1
    out, lse = torch.full((10, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((10, 4), 7.0, device="cuda")
    o, l, _ = B.call(algo=algo, Q=Q, out=out, lse=lse)
    assert o is out and l is lse
    B.check(out, lse, Q=Q)
    for t in (out, lse):
        assert bool((t[:1] == 7).all()) and bool((t[7:] == 7).all())
    # of a sequence with more than max_q queries the first max_q are computed
    out.fill_(7.0)
    B.call(algo=algo, Q=Q, out=out, max_q=2)
    assert bool((out[3:5] == 7).all()) and bool((out[1:3] != 7).any())
    B.check(out, Q=Q, seqs=[1])


@both
@pytest.mark.parametrize("window", [0, 17])
def test_max_q_keeps_the_positions(window, algo):
    """The first max_q queries of a sequence keep the keys that they keep without the bound."""
    B = Batch([50, 300, 3], [40, 2, 9], 4, 2, 64, 16)
    out, lse = torch.full_like(B.Q, 7.0), torch.full((51, 4), 7.0, device="cuda")
    B.call(algo=algo, window=window, max_q=5, out=out, lse=lse)
    Q, got, gl = (t.double().cpu().numpy() for t in (B.Q, out, lse))
    for b, (S, n) in enumerate(zip(B.lens, B.qs)):
        q0, k = int(B.offsets[b]), min(n, 5)
        want, wl, tol, lt = kv.attention(Q[q0:q0 + k], *B.values(b), 64 ** -0.5, kv.keeps(S, n, True, window)[:k], HALF["bf16"])
        assert np.all(np.abs(got[q0:q0 + k] - want) <= tol)
        none = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl[q0:q0 + k]), none)
        assert np.all(np.abs(gl[q0:q0 + k][~none] - wl[~none]) <= lt[~none])
        assert np.all(got[q0 + k:q0 + n] == 7) and np.all(gl[q0 + k:q0 + n] == 7)


@both
def test_max_kv_bounds_the_lengths(algo):
    B = Batch([100, 40], [1, 1], 4, 1, 128, 16)
    out, _, _ = B.call(algo=algo, max_kv=64)
    C = Batch([100, 40], [1, 1], 4, 1, 128, 16)
    C.lens, C.slots = [64, 40], [C.slots[0][:64], C.slots[1]]
    C.check(out)


@both
def test_pages_that_are_not_there(algo):
    """Tokens of a page outside [0, pages) count for no row."""
    B = Batch([200, 90], [2, 1], 4, 2, 128, 32)
    pages = B.cache.k_codes.shape[0]
    gone = {0: [0, 3], 1: [1]}
    k = [B.values(b) for b in range(2)]
    for b, ps in gone.items():
        for i, p in enumerate(ps):
            B.table[b, p] = [-1, pages, 1 << 30, -(1 << 31)][(i + b) % 4]
    out, lse, _ = B.call(algo=algo, with_lse=True)
    Q = B.Q.double().cpu().numpy()
    for b in range(2):
        keep = kv.keeps(B.lens[b], B.qs[b], True, 0)
        for p in gone[b]:
            keep[:, p * 32:(p + 1) * 32] = False
        q0 = int(B.offsets[b])
        want, wl, tol, lt = kv.attention(Q[q0:q0 + B.qs[b]], *k[b], 128 ** -0.5, keep, HALF["bf16"])
        got, gl = out[q0:q0 + B.qs[b]].double().cpu().numpy(), lse[q0:q0 + B.qs[b]].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol) and np.all(np.abs(gl - wl) <= lt)
    B.table[:] = -1
    out, lse, _ = B.call(algo=algo, with_lse=True)
    assert int(out.count_nonzero()) == 0 and bool(torch.isneginf(lse).all())


@both
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-6, 1.0, 30.0])
def test_scales(scale, algo):
    B = Batch([150, 33], [3, 1], 4, 2, 64, 16, x="f16")
    out, lse, _ = B.call(algo=algo, scale=scale, with_lse=True)
    B.check(out, lse, scale=scale)


@both
@pytest.mark.parametrize("size", [1e-38, 1e-20, 1e-4, 300.0, 1e6, 1e30])
def test_queries_of_any_size(size, algo):
    """bf16 queries of any magnitude: logits next to nothing, or one key alone."""
    B = Batch([130, 40], [2, 1], 4, 2, 96, 16)
    Q = (B.Q.float() * size).to(torch.bfloat16)
    Q[0, 0, ::3] = 0
    Q[1, 1, :] = 0
    if size < 1e20:
        out, lse, _ = B.call(algo=algo, Q=Q, with_lse=True)
        B.check(out, lse, Q=Q)
    else:
        out, lse, _ = B.call(algo=algo, Q=Q, with_lse=True, scale=1e-30)
        B.check(out, lse, Q=Q, scale=1e-30)


@both
def test_a_row_that_is_not_finite_touches_no_other(algo):
    B = Batch([130, 40], [2, 1], 8, 2, 128, 16)
    want, _, _ = B.call(algo=algo)
    Q = B.Q.clone()
    Q[0, 1, 5], Q[1, 6, 0], Q[2, 3, 127] = float("nan"), float("inf"), float("-inf")
    out, _, _ = B.call(algo=algo, Q=Q)
    hit = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 6] = hit[2, 3] = True
    assert torch.equal(out[~hit], want[~hit]) and bool(out[0, 1].isnan().all())


@both
@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_flat_and_sharp_rows(spread, algo):
    """Every key alike, and rows where the largest logit grows by hundreds along the sequence."""
    B = Batch([600, 257], [1, 4], 6, 2, 128, 64, spread=spread)
    out, lse, _ = B.call(algo=algo, with_lse=True)
    B.check(out, lse)


@both
def test_growing_logits(algo):
    """Keys ordered so that the reference is raised in nearly every tile."""
    B = Batch([512], [1], 4, 1, 64, 16)
    K = torch.linspace(0, 2.6, 512, device="cuda")[:, None, None] * torch.ones(512, 1, 64, device="cuda")
    ssn.kv_nvfp4_append(K, torch.randn(512, 1, 64, device="cuda"), B.dev(B.slots[0]), B.cache)
    B.Q = torch.ones_like(B.Q) * torch.tensor([1.0, -1.0, 4.0, -4.0], device="cuda", dtype=B.Q.dtype)[:, None]
    out, lse, _ = B.call(algo=algo, with_lse=True)
    B.check(out, lse)


@both
@pytest.mark.parametrize("D,Hq,H,n,window", [(128, 16, 2, 1, 0), (64, 4, 4, 1, 0), (256, 8, 1, 1, 0), (128, 10, 2, 9, 0),
                                             (160, 3, 1, 2, 3000), (128, 8, 1, 1, 700)])
def test_long_sequences_are_split(D, Hq, H, n, window, algo):
    B = Batch([9001, 4100], [n, n], Hq, H, D, 64)
    out, lse, _ = B.call(algo=algo, uniform=True, with_lse=True, window=window)
    B.check(out, lse, window=window)
    again, lse2, _ = B.call(algo=algo, uniform=True, with_lse=True, window=window)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@both
def test_split_with_short_sequences_among_long(algo):
    """Splits that get no keys of a sequence."""
    B = Batch([5000, 1, 0, 40, 700], [1, 1, 1, 1, 1], 8, 1, 128, 16)
    out, lse, _ = B.call(algo=algo, uniform=True, with_lse=True)
    B.check(out, lse)


@pytest.mark.parametrize("B", [2, 63, 64, 65, 200, 256, 257])
@pytest.mark.parametrize("window", [0, 2500])
def test_batches_with_one_long_sequence(B, window):
    """Parts of equal work: some sequences end and others begin inside one, and some have no keys or no query."""
    rng = np.random.default_rng(B + window)
    lens = [int(n) for n in rng.integers(0, 70, B)]
    lens[B // 2], lens[0] = 4321, 0
    qs = [int(q) for q in rng.integers(0, 2, B)]
    qs[B // 2] = qs[0] = 1
    X = Batch(lens, qs, 4, 1, 64, 16, seed=B)
    out, lse, _ = X.call(with_lse=True, window=window, max_q=1)
    X.check(out, lse, window=window)


def test_batches_without_a_query():
    X = Batch([3000, 2500], [0, 0], 8, 2, 128, 16)
    out, _, _ = X.call(max_q=1, max_kv=3000)
    assert out.shape == (0, 8, 128)
    X = Batch([3000, 2500, 10], [0, 1, 0], 8, 2, 128, 16)
    out, lse, _ = X.call(max_q=1, with_lse=True)
    X.check(out, lse)


@both
def test_strided_queries(algo):
    B = Batch([90, 30], [3, 2], 4, 2, 96, 16)
    wide = torch.zeros(5, 12, 96, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:7] = B.Q
    want, _, _ = B.call(algo=algo)
    out, _, _ = B.call(algo=algo, Q=wide[:, 3:7])
    assert torch.equal(out, want) and out.is_contiguous()
    out, _, _ = B.call(algo=algo, Q=B.Q.transpose(0, 1).contiguous().transpose(0, 1))
    assert torch.equal(out, want)


@both
def test_offsets_beyond_32_bits(algo):
    H, D, page = 8, 256, 256
    pages = (1 << 32) // (H * page * D // 2) + 8
    B = Batch([300], [1], 8, H, D, page)
    ts = B.cache.k_tensor_scale, B.cache.v_tensor_scale
    big = ssn.kv_nvfp4_empty(pages, page, D, *ts)
    for i, p in enumerate(B.table[0, :2]):
        for s, d in zip(B.cache[:4], big[:4]):
            d[pages - 1 - i] = s[int(p)]
    want, _, _ = B.call(algo=algo)
    small, B.cache = B.cache, big
    B.table[0, :2] = [pages - 1, pages - 2]
    out, _, _ = B.call(algo=algo)
    assert torch.equal(out, want)


def test_captured_and_replayed_beside_another():
    """Two captured calls with workspaces of their own; lengths, pages and queries of the replay's time."""
    A, B = Batch([4000, 2500], [1, 1], 8, 1, 128, 16, seed=1), Batch([3000], [2], 4, 1, 64, 16, seed=2)
    st = []
    for X in (A, B):
        t = dict(Q=X.Q, table=X.dev(X.table), lens=X.dev(np.int32(X.lens)), out=torch.zeros_like(X.Q))
        t["args"] = (t["Q"], X.cache, t["table"], t["lens"])
        t["kw"] = dict(out=t["out"], max_kv=4096 if X.table.shape[1] * 16 >= 4096 else None)
        ssn.attn_kv_nvfp4(*t["args"], **t["kw"])
        st.append(t)
    torch.cuda.synchronize()
    graphs = []
    for t in st:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ssn.attn_kv_nvfp4(*t["args"], **t["kw"])
        graphs.append(g)
    side = torch.cuda.Stream()
    for i in range(4):
        for X, t in zip((A, B), st):
            t["Q"].copy_(torch.randn_like(t["Q"]))
            t["lens"].copy_(torch.tensor([n - 700 * i for n in X.lens], dtype=torch.int32))
            t["out"].zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for t in st:
            got = t["out"].clone()
            want, _, _ = ssn.attn_kv_nvfp4(*t["args"], max_kv=t["kw"]["max_kv"])
            assert torch.equal(got, want)


def test_two_calls_on_two_streams():
    A, B = Batch([6000], [1], 8, 1, 128, 16, seed=3), Batch([7000], [1], 8, 1, 128, 16, seed=4)
    want = [X.call()[0].clone() for X in (A, B)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for X, s in zip((A, B), streams):
            with torch.cuda.stream(s):
                got.append(X.call()[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_prepared_call():
    B = Batch([600, 90], [1, 1], 8, 2, 128, 16)
    want, _, _ = B.call()
    call, (out, _, used) = B.call(prepare=True)
    call(); call()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and used.value == ssn.ALGO_STREAM


def test_a_model_decodes():
    """A prompt and six decoded tokens through append and attention, as a layer uses them: every step equals attention
    over what the cache holds."""
    torch.manual_seed(5)
    Hq, H, D, page, pages = 8, 2, 64, 16, 12
    ts = torch.full((H,), 4.5 / 2688, device="cuda")
    cache = ssn.kv_nvfp4_empty(pages, page, D, ts, ts)
    for t in cache[:4]:
        t.fill_(0xFF)
    table = torch.randperm(pages, device="cuda").to(torch.int32).view(2, 6)
    lens = torch.tensor([37, 20], device="cuda", dtype=torch.int32)
    offsets = torch.tensor([0, 37, 57], device="cuda", dtype=torch.int32)
    done = torch.zeros(2, dtype=torch.int64)
    for step in range(7):
        qs = [37, 20] if step == 0 else [1, 1]
        qkv = torch.randn(sum(qs), Hq + 2 * H, D, device="cuda").to(torch.bfloat16)
        slots = torch.cat([table[b].long()[(p := torch.arange(int(done[b]), int(done[b]) + qs[b], device="cuda")) // page]
                           * page + p % page for b in range(2)])
        done += torch.tensor(qs)
        ssn.kv_nvfp4_append(qkv[:, Hq:Hq + H], qkv[:, Hq + H:], slots, cache)
        if step:
            lens += 1
        out, _, _ = ssn.attn_kv_nvfp4(qkv[:, :Hq], cache, table, lens, offsets if step == 0 else None,
                                      max_q=max(qs))
        at = 0
        for b in range(2):
            S, n = int(done[b]), qs[b]
            j = torch.arange(S, device="cuda")
            K, V = ssn.kv_nvfp4_read(table[b].long()[j // page] * page + j % page, cache, out_dtype=torch.float32)
            want, _, tol, _ = kv.attention(qkv[at:at + n, :Hq].double().cpu().numpy(), K.double().cpu().numpy(),
                                           V.double().cpu().numpy(), D ** -0.5, kv.keeps(S, n, True, 0), 2.0 ** -8)
            # K and V were read back rounded to f32: half a step more of every logit and value, of which the bound counts many
            assert np.all(np.abs(out[at:at + n].double().cpu().numpy() - want) <= tol)
            at += n


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("Hq,H,lens,qs", [(1, 1, [300, 129, 128, 127], [300, 129, 1, 127]),
                                          (5, 1, [64, 65, 200], [64, 33, 77]), (16, 2, [150, 40], [60, 40]),
                                          (6, 6, [131], [131])])
def test_prompts(D, Hq, H, lens, qs):
    """Whole prompts and chunks, of one query head to a key head up to eight; rows over several workgroups."""
    B = Batch(lens, qs, Hq, H, D, [16, 32, 48, 64, 128][(D // 32 + Hq) % 5], x="f16" if D % 64 else "bf16")
    out, lse, used = B.call(with_lse=True)
    assert used == (TILE if max(qs) * (Hq // H) > (32 if D > 128 else 64) else STREAM)
    B.check(out, lse)


@pytest.mark.parametrize("window", [1, 31, 33, 64, 100, 129])
@pytest.mark.parametrize("D,Hq", [(64, 1), (128, 3), (256, 2)])
def test_prompts_with_a_window(D, Hq, window):
    B = Batch([333, 70], [333, 20], Hq, 1, D, 16)
    out, lse, _ = B.call(with_lse=True, window=window)
    B.check(out, lse, window=window)


def test_chunk_after_a_long_context():
    """Few rows and many keys: the tiles split too."""
    B = Batch([6000, 2100], [30, 25], 8, 2, 128, 32)
    out, lse, used = B.call(with_lse=True)
    assert used == TILE and ssn.lib().attn_kv_nvfp4_workspace_bytes(2, 8, 2, 128, 30, 6000) > 0
    B.check(out, lse)
    again, _, _ = B.call()
    assert torch.equal(out, again)


def test_both_ways_agree():
    """The two kernels differ by the roundings of their sums alone: far less than a step of bf16 of the largest value."""
    B = Batch([700, 300, 90], [40, 3, 90], 12, 4, 96, 48)
    a, la, _ = B.call(algo=STREAM, out_dtype=torch.float32, with_lse=True)
    b, lb, _ = B.call(algo=TILE, out_dtype=torch.float32, with_lse=True)
    # each is within its bound of the same value: terms of 2^-11, sums of f32
    B.check(a, la, out_type="f32")
    B.check(b, lb, out_type="f32")
    assert float((a - b).abs().max()) <= 2 * 2.0 ** -10 * float(a.abs().max())


@pytest.mark.parametrize("B", [1, 2, 5, 64, 65, 130, 4097])
@pytest.mark.parametrize("uniform", [False, True])
def test_a_bound_of_queries_far_above_them(B, uniform):
    """max_q = 2^28, of which no launch could hold the rows: workgroups for the queries there are."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90 if B > 200 else 400, B)
    qs = np.full(B, 7) if uniform else rng.integers(0, 5 if B > 200 else 70, B)
    if not uniform and B > 2:
        qs[0], qs[1], qs[-1], lens[-1] = 0, 150, 3, 200
    X = Batch(lens.tolist(), qs.tolist(), 4, 1, 64, 16, seed=B)
    for algo in (ssn.ALGO_AUTO, TILE):
        out, lse, used = X.call(algo=algo, uniform=uniform, max_q=1 << 28, with_lse=True)
        assert used == TILE
        X.check(out, lse, seqs=range(0, B, 1 + B // 130))


def test_a_large_batch_without_its_bound():
    """2048 sequences of a few queries, 64 key heads: by default max_q is the number of all queries. Rows before the first
    and behind the last sequence are left."""
    B, H, D = 2048, 64, 32
    rng = np.random.default_rng(9)
    qs = rng.integers(0, 9, B)
    X = Batch([5] * B, qs.tolist(), H, H, D, 16)
    T = int(qs.sum())
    assert B * H * (-(-(T + 24) // 128)) > 1 << 23
    Q = torch.cat([X.Q[:16], X.Q, X.Q[:8]])
    X.offsets = X.offsets + 16
    out, lse = torch.full((T + 24, H, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T + 24, H), 7.0, device="cuda")
    _, _, used = X.call(Q=Q, out=out, lse=lse, max_q=None)
    assert used == TILE
    X.check(out, lse, Q=Q, seqs=range(0, B, 97))
    for t in (out, lse):
        assert bool((t[:16] == 7).all()) and bool((t[-8:] == 7).all())
    want, wl, used = X.call(Q=Q, max_q=8, with_lse=True)
    assert used == STREAM
    # Both kernels are within their bound of one value. Values: terms of 2^-11 each and half a step of bf16, of at most 2688 s_h < 6.
    # Logarithms: a logit has D + 24 steps of 2^-23 of at most 16 (scale sum |q k| log2 e), that is 2^-13 of both at most.
    a, b, la, lb = out[16:-8].float(), want[16:-8].float(), lse[16:-8], wl[16:-8]
    assert float((a - b).abs().max()) <= 2 * (2.0 ** -11 + 2.0 ** -8) * 6
    assert torch.equal(torch.isneginf(la), torch.isneginf(lb))
    assert float((la - lb).nan_to_num(0).abs().max()) <= 2.0 ** -13


@pytest.mark.parametrize("D,rows,algo", [(64, 96, STREAM), (64, 97, TILE), (96, 96, STREAM), (128, 96, STREAM), (128, 97, TILE),
                                         (160, 32, STREAM), (160, 33, TILE), (256, 32, STREAM), (256, 33, TILE)])
@pytest.mark.parametrize("n", [1, 2])
def test_where_the_choice_changes(D, rows, algo, n):
    """96 rows to a key head (32 beyond a width of 128) are streamed, more are tiles: right on both sides."""
    if rows % n:
        rows += 1 if algo == TILE else -1
    B = Batch([150, 37, 0], [n, n, n], rows // n, 1, D, 16)
    out, lse, used = B.call(with_lse=True)
    assert used == algo
    B.check(out, lse)


@both
@pytest.mark.parametrize("S,parts", [(2000, (2, 16)), (6000, (17, 64)), (12000, (65, 256))])
@pytest.mark.parametrize("D", [32, 96, 192, 224])
def test_joins_of_every_width(D, S, parts, algo):
    """The three forms of the join, where a row's four-value pieces do not divide the lanes that share it."""
    H, n = 1, 2
    B = Batch([S], [n], 2, H, D, 16)
    # both kernels split alike here, and the tiles' 128 rows make the larger workspace
    count = ssn.lib().attn_kv_nvfp4_workspace_bytes(1, 2, H, D, n, B.table.shape[1] * 16) // (128 * (D + 2) * 4)
    assert parts[0] <= count <= parts[1]
    out, lse, _ = B.call(algo=algo, with_lse=True)
    B.check(out, lse)
