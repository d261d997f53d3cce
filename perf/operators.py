"""The measured cases of the 4-bit integer products and of the token permutation.

Five operators, as a mixture-of-experts model with integer 4-bit weights uses them:

* ``gemv``     Y = X . W_hat^T for a few rows of X, W_hat[n, k] = s[n, g] * (q[n, k] - z[n, g]), codes of 4
               bits, one scale and one zero point per group of consecutive k (``gemv_int4``);
* ``experts``  the same product for the rows of every expert, plain or with the SiLU gate
               (``moe_grouped_gemv_int4``);
* ``weights``  4-bit codes, scales and zero points from float weights and back (``int4_quantize``,
               ``int4_dequantize``);
* ``permute``  tokens copied to expert order, and its gradient (``moe_permute``, ``moe_permute_backward``);
* ``unpermute`` expert rows added back with the routing weights, and its gradient (``moe_unpermute``,
               ``moe_unpermute_backward``).

A case is a dict of plain values. ``run`` computes it with elementary torch operations in 32 bits, or, where
``own`` is true, with the calls above.
"""
import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one linear layer of a small test model at one token: the call's latency
        dict(name="gemv-small", kind="gemv", M=1, N=256, K=512, group=64, asym=False, x="f16", s="f16", y="f16"),
        # an up projection of a 5120-wide model at one decoded token
        dict(name="gemv-decode", kind="gemv", M=1, N=13824, K=5120, group=128, asym=True, x="bf16", s="bf16", y="f32"),
        # the output head of that model for eight sequences
        dict(name="gemv-head", kind="gemv", M=8, N=131072, K=5120, group=128, asym=True, x="bf16", s="f16", y="f32"),
        # a batch of sequences on a layer of odd sizes, whose last group is half a group
        dict(name="gemv-ragged", kind="gemv", M=50, N=4097, K=5152, group=64, asym=True, x="f16", s="f16", y="f16"),
        # gate and up projections of ten experts at one decoded token
        dict(name="experts-up", kind="experts", T=1, k=10, E=512, N=1024, K=2048, group=128, asym=True, silu=True,
             hot=False, x="bf16", s="bf16", y="bf16"),
        # down projections at 32 tokens, rows already in expert order
        dict(name="experts-down", kind="experts", T=32, k=10, E=512, N=2048, K=512, group=64, asym=False, silu=False,
             hot=False, x="bf16", s="bf16", y="f32"),
        # a layer's float weights to 4 bits and back
        dict(name="weights-layer", kind="weights", N=13824, K=5120, group=128, asym=True, w="f32", s="bf16"),
        # a small ragged one, symmetric
        dict(name="weights-ragged", kind="weights", N=255, K=2080, group=64, asym=False, w="bf16", s="f16"),
        # a prompt of 4096 tokens to expert order
        dict(name="permute-prompt", kind="permute", back=False, T=4096, k=10, E=512, D=2048, drop=0, weighted=False,
             x="bf16", y="bf16"),
        # the gradient of a weighted permutation of odd width, some entries dropped
        dict(name="permute-grad", kind="permute", back=True, T=511, k=6, E=64, D=1001, drop=37, weighted=True,
             x="f32", y="f32"),
        # eight decoded tokens back from expert order
        dict(name="unpermute-decode", kind="unpermute", back=False, T=8, k=10, E=512, D=2048, drop=0, weighted=True,
             x="bf16", y="bf16"),
        # the gradient of a prompt's weighted sum: expert rows and routing weights
        dict(name="unpermute-grad", kind="unpermute", back=True, T=4096, k=10, E=512, D=2048, drop=0, weighted=True,
             x="bf16", y="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["gemv", "experts", "weights", "permute", "unpermute"])
    t16 = ["bf16", "f16"]
    if kind in ("gemv", "experts"):
        x = rng.choice(t16)
        out = dict(kind=kind, asym=rng.random() < 0.5, x=x, s=rng.choice(t16), y=rng.choice(["f32", x]))
        K = 32 * _log(rng, 2, 256)
        out.update(K=K, group=rng.choice([32, 64, 128, 128, 32 * rng.randint(1, 12), K]))
    if kind == "gemv":
        # up to the output head's work: N K weights and M N K products
        M = _log(rng, 1, 64)
        out.update(M=M, N=_log(rng, 64, min(131072, (8 * 131072 * 5120) // (max(M, 8) * K))))
        return out
    if kind == "experts":
        E = _log(rng, 4, 512)
        hot = rng.random() < 0.3
        out.update(T=_log(rng, 1, 48), k=rng.randint(1, min(10, E // (2 if hot else 1))), E=E, hot=hot,
                   silu=rng.random() < 0.5, N=2 * _log(rng, 32, min(2048, 512 * 1024 * 2048 // (2 * E * K))))
        return out
    if kind == "weights":
        K = 32 * _log(rng, 2, 256)
        return dict(kind=kind, N=_log(rng, 16, 13824 * 5120 // K), K=K, asym=rng.random() < 0.5,
                    group=rng.choice([32, 64, 128, 256, 32 * rng.randint(1, 12), K]), w=rng.choice(list(_TYPES)),
                    s=rng.choice(t16))
    E, x = _log(rng, 4, 512), rng.choice(list(_TYPES))
    T, k = _log(rng, 1, 4096), rng.randint(1, min(10, E))
    # up to a prompt's bytes in bf16, also where the rows are f32
    D = _log(rng, 64, min(8192, 4096 * 10 * 2048 // (T * k) // (2 if x == "f32" else 1)))
    return dict(kind=kind, back=rng.random() < 0.5, T=T, k=k, E=E, D=D,
                drop=rng.choice([0, 0, rng.randint(0, T * k // 8)]), weighted=rng.random() < 0.7, x=x,
                y="f32" if kind == "unpermute" and rng.random() < 0.3 else x)


# ------------------------------------------------------------------------------------------------
# inputs


def _codes(g, shape, K):
    """Packed 4-bit codes [*shape, K/2], bell-shaped about 7.5 as quantised weights are."""
    out = torch.empty((*shape, K // 2), dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        q = torch.randn((2, part.numel()), generator=g, device="cuda").mul_(2.6).add_(7.5).round_().clamp_(0, 15)
        q = q.to(torch.uint8)
        part.copy_(q[0] | (q[1] << 4))
    return out


def _weights4(case, g, lead):
    N, K = case["N"], case["K"]
    groups = -(-K // case["group"])
    codes = _codes(g, (*lead, N), K)
    # a group's scale is its range over fifteen steps: some 0.02 * 5 / 15, varying by a factor of two or so
    scales = (torch.randn((*lead, N, groups), generator=g, device="cuda").mul_(0.3).exp_().mul_(0.007))
    zeros = None
    if case["asym"]:
        zeros = torch.randint(5, 11, (*lead, N, groups), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales.to(_TYPES[case["s"]]), zeros


def _ids(case, g):
    """Expert ids [T, k], distinct in a token; `hot` routings crowd onto the first 2k experts."""
    T, k = case["T"], case["k"]
    E = 2 * k if case.get("hot") else case["E"]
    return torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices


def _route(ids, E, drop, g):
    """(offsets [E+1], row_token [R], row_of [T k]) of the flat entries grouped by expert; `drop` of them get
    no row (-1)."""
    T, k = ids.shape
    flat = ids.reshape(-1).clone()
    if drop:
        flat[torch.randperm(T * k, generator=g, device="cuda")[:drop]] = E
    order = torch.sort(flat, stable=True).indices
    R = T * k - drop
    row_of = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    row_of[order[:R]] = torch.arange(R, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
    return offsets, (order[:R] // k).to(torch.int32), row_of


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, t):
        return torch.randn(shape, generator=g, device="cuda").to(_TYPES[t])

    st = dict(case=dict(case))
    kind = case["kind"]
    if kind == "gemv":
        st["X"] = normal((case["M"], case["K"]), case["x"])
        st["codes"], st["scales"], st["zeros"] = _weights4(case, g, ())
    elif kind == "experts":
        ids = _ids(case, g)
        st["offsets"], row_token, _ = _route(ids, case["E"], 0, g)
        st["R"] = case["T"] * case["k"]
        # gate and up gather their tokens; the down projection's rows are in expert order already
        st["row_token"] = row_token if case["silu"] else None
        st["X"] = normal((case["T"] if case["silu"] else st["R"], case["K"]), case["x"])
        st["codes"], st["scales"], st["zeros"] = _weights4(case, g, (case["E"],))
    elif kind == "weights":
        # rows of different spread, as the layers of a model have
        spread = torch.randn((case["N"], 1), generator=g, device="cuda").mul_(0.3).exp_().mul_(0.02)
        st["W"] = torch.randn((case["N"], case["K"]), generator=g, device="cuda").mul_(spread).to(_TYPES[case["w"]])
    else:
        T, k, D = case["T"], case["k"], case["D"]
        _, _, st["row_of"] = _route(_ids(case, g), case["E"], case["drop"], g)
        st["R"] = T * k - case["drop"]
        st["weights"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1) if case["weighted"] else None
        if kind == "permute":
            st["X"] = normal((T, D), case["x"])
            if case["back"]:
                st["dXp"] = normal((st["R"], D), case["x"])
        else:
            st["Yp"] = normal((st["R"], D), case["x"])
            if case["back"]:
                st["dout"] = normal((T, D), case["y"])
    return st


# ------------------------------------------------------------------------------------------------
# one pass


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["kind"]](state, state["case"])


def _run_own(st):
    import structured_sparse_nvfp4_amd as ssn
    c = st["case"]
    kind = c["kind"]
    if kind == "gemv":
        return ssn.gemv_int4(st["X"], st["codes"], st["scales"], st["zeros"], group=c["group"],
                             y_dtype=_TYPES[c["y"]])[0]
    if kind == "experts":
        return ssn.moe_grouped_gemv_int4(st["X"], st["row_token"], st["offsets"], st["R"], st["codes"], st["scales"],
                                         st["zeros"], group=c["group"],
                                         epilogue=ssn.EPI_SILU_GATE if c["silu"] else ssn.EPI_NONE,
                                         y_dtype=_TYPES[c["y"]])[0]
    if kind == "weights":
        codes, scales, zeros = ssn.int4_quantize(st["W"], group=c["group"], symmetric=not c["asym"],
                                                 scale_dtype=_TYPES[c["s"]])
        W = ssn.int4_dequantize(codes, scales, zeros, group=c["group"])
        return (W, scales, zeros) if c["asym"] else (W, scales)
    if kind == "permute":
        if not c["back"]:
            return ssn.moe_permute(st["X"], st["row_of"], st["weights"], R=st["R"])
        X = st["X"] if c["weighted"] else None
        dX, dw = ssn.moe_permute_backward(st["dXp"], st["row_of"], c["T"], st["weights"], X=X)
        return (dX, dw) if c["weighted"] else dX
    if not c["back"]:
        return ssn.moe_unpermute(st["Yp"], st["row_of"], c["T"], st["weights"], out_dtype=_TYPES[c["y"]])
    Yp = st["Yp"] if c["weighted"] else None
    dYp, dw = ssn.moe_unpermute_backward(st["dout"], st["row_of"], st["R"], st["weights"], Yp=Yp,
                                         y_dtype=_TYPES[c["x"]])
    return (dYp, dw) if c["weighted"] else dYp


def _unpack(codes):
    """[..., K/2] bytes -> [..., K] codes, the low nibble first."""
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _spread(v, group, K):
    """One value per group -> one per k."""
    return v[..., torch.arange(K, device="cuda") // group]


def _decode(codes, scales, zeros, group):
    q = _unpack(codes).float()
    K = q.shape[-1]
    z = 8.0 if zeros is None else _spread(zeros.float(), group, K)
    return (q - z) * _spread(scales.float(), group, K)


def _plain_gemv(st, c):
    W = _decode(st["codes"], st["scales"], st["zeros"], c["group"])
    return (st["X"].float() @ W.t()).to(_TYPES[c["y"]])


def _plain_experts(st, c):
    R = st["R"]
    expert = torch.searchsorted(st["offsets"][1:].contiguous(), torch.arange(R, dtype=torch.int32, device="cuda"),
                                right=True)
    X = st["X"].float()
    if st["row_token"] is not None:
        X = X[st["row_token"].long()]
    parts = []
    for r in range(0, R, 64):      # 64 rows' weights at a time
        e = expert[r:r + 64]
        W = _decode(st["codes"][e], st["scales"][e], None if st["zeros"] is None else st["zeros"][e], c["group"])
        parts.append((W @ X[r:r + 64, :, None])[..., 0])
    Y = torch.cat(parts)
    if c["silu"]:
        gate, up = Y.chunk(2, 1)
        Y = gate / (1.0 + torch.exp(-gate)) * up
    return Y.to(_TYPES[c["y"]])


def _plain_weights(st, c):
    """Scale, zero point and codes per group; quotients in 64 bits, where their rounding borders lie."""
    N, K, group = c["N"], c["K"], c["group"]
    groups = -(-K // group)
    W = torch.zeros((N, groups * group), dtype=torch.float64, device="cuda")
    W[:, :K] = st["W"].double()
    W = W.view(N, groups, group)
    t = _TYPES[c["s"]]
    if c["asym"]:
        lo, hi = W.amin(2).clamp(max=0.0), W.amax(2).clamp(min=0.0)
        scales = ((hi - lo) / 15.0).clamp(max=torch.finfo(t).max).float().to(t)
        s = scales.double()
        safe = torch.where(s > 0, s, 1.0)
        z = torch.where(s > 0, (-lo / safe).round().clamp(0.0, 15.0), 0.0)
        q = ((W / safe[..., None]).round() + z[..., None]).clamp(0.0, 15.0)
    else:
        scales = (W.abs().amax(2) / 7.0).clamp(max=torch.finfo(t).max).float().to(t)
        s = scales.double()
        safe = torch.where(s > 0, s, 1.0)
        z = torch.full_like(s, 8.0)
        q = ((W / safe[..., None]).round() + 8.0).clamp(0.0, 15.0)
    q = torch.where(s[..., None] > 0, q, z[..., None])
    What = ((q - z[..., None]) * s[..., None]).view(N, groups * group)[:, :K].float()
    return (What, scales, z.to(torch.uint8)) if c["asym"] else (What, scales)


def _rows(st, c):
    """(row of every (token, slot), one past the last where it has none; whether it has one)."""
    row = st["row_of"].view(c["T"], c["k"]).long()
    has = row >= 0
    return torch.where(has, row, st["R"]), has


def _plain_permute(st, c):
    if c["back"]:
        dX, dw = _gather(st["dXp"], st, c, st["X"])
        return (dX.to(_TYPES[c["x"]]), dw) if c["weighted"] else dX.to(_TYPES[c["x"]])
    return _scatter(st["X"], st, c)


def _plain_unpermute(st, c):
    if not c["back"]:
        return _gather(st["Yp"], st, c, None)[0].to(_TYPES[c["y"]])
    dYp = _scatter(st["dout"], st, c)
    return (dYp, _gather(st["Yp"], st, c, st["dout"])[1]) if c["weighted"] else dYp


def _scatter(A, st, c):
    """B[row] = weight * A[token], in the rows' type; entries without a row go to one behind the last."""
    row, _ = _rows(st, c)
    B = torch.empty((st["R"] + 1, c["D"]), dtype=_TYPES[c["x"]], device="cuda")
    A = A.float()
    for j in range(c["k"]):
        B[row[:, j]] = (A * st["weights"][:, j, None] if c["weighted"] else A).to(B.dtype)
    return B[:-1]


def _gather(B, st, c, A):
    """(sum over the slots of weight * B[row], the slots' products <A[token], B[row]> if A is given)."""
    row, has = _rows(st, c)
    out = torch.zeros((c["T"], c["D"]), device="cuda")
    dw = []
    for j in range(c["k"]):
        b = torch.where(has[:, j, None], B[row[:, j].clamp(max=st["R"] - 1)].float(), 0.0)
        out = out + (b * st["weights"][:, j, None] if c["weighted"] else b)
        if A is not None:
            dw.append((b * A.float()).sum(1))
    return out, torch.stack(dw, 1) if dw else None


_PLAIN = {"gemv": _plain_gemv, "experts": _plain_experts, "weights": _plain_weights, "permute": _plain_permute,
          "unpermute": _plain_unpermute}


# ------------------------------------------------------------------------------------------------
# the bytes and operations a pass cannot do without


def _weight_bytes(c, rows):
    groups = -(-c["K"] // c["group"])
    return rows * (c["K"] / 2 + groups * (3 if c["asym"] else 2))


def work(case):
    c = case
    kind = c["kind"]
    if kind == "gemv":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": _weight_bytes(c, N) + M * K * 2 + M * N * _BYTES[c["y"]], "flops": 2.0 * M * N * K}
    if kind == "experts":
        # the experts that a routing touches: T draws of k distinct ones
        R, N, K = c["T"] * c["k"], c["N"], c["K"]
        pool = 2 * c["k"] if c["hot"] else c["E"]
        touched = pool * (1.0 - (1.0 - c["k"] / pool) ** c["T"])
        rows = c["T"] if c["silu"] else R
        return {"bytes": _weight_bytes(c, touched * N) + rows * K * 2 + R * (N // 2 if c["silu"] else N) * _BYTES[c["y"]]
                + (c["E"] + 1) * 4 + (R * 4 if c["silu"] else 0), "flops": 2.0 * R * N * K}
    if kind == "weights":
        # read the float weights, write the packed form, read it, write 32-bit weights
        N, K = c["N"], c["K"]
        return {"bytes": N * K * _BYTES[c["w"]] + 2 * _weight_bytes(c, N) + N * K * 4, "flops": 6.0 * N * K}
    T, k, D = c["T"], c["k"], c["D"]
    R = T * k - c["drop"]
    index = T * k * (4 + (4 if c["weighted"] else 0))
    ex, ey = _BYTES[c["x"]], _BYTES[c["y"]]
    # rows on the token side: one of the token's own type, and a second where the weights' gradient needs it
    token = T * D * (ey if kind == "unpermute" else ex)
    rows = R * D * ex
    grad = c["back"] and c["weighted"]
    if grad:
        if kind == "permute":
            token += T * D * ex
        else:
            rows += R * D * ex
    return {"bytes": token + rows + index + (T * k * 4 if grad else 0),
            "flops": R * D * ((2.0 if c["weighted"] else 1.0) + (2.0 if grad else 0.0))}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_product(X, codes, scales, zeros, group):
    """sum over the groups of s[n, g] * sum over the group's k of x (q - z)."""
    M, K = X.shape
    Y = torch.zeros((M, codes.shape[0]), dtype=torch.float64, device="cuda")
    for g, k0 in enumerate(range(0, K, group)):
        k1 = min(K, k0 + group)
        part = codes[:, k0 // 2:k1 // 2].to(torch.int64)
        even, odd = (part % 16).double(), (part // 16).double()
        xe, xo = X[:, k0:k1:2].double(), X[:, k0 + 1:k1:2].double()
        z = zeros[:, g].double() if zeros is not None else torch.full_like(scales[:, g], 8, dtype=torch.float64)
        dot = xe @ even.t() + xo @ odd.t() - X[:, k0:k1].double().sum(1)[:, None] * z
        Y += dot * scales[:, g].double()
    return Y


def exact(case, seed):
    st = prepare(case, seed)
    kind, c = case["kind"], case
    if kind == "gemv":
        return _exact_product(st["X"], st["codes"], st["scales"], st["zeros"], c["group"])
    if kind == "experts":
        off = st["offsets"].tolist()
        Y = torch.zeros((st["R"], c["N"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            if a < b:
                x = st["X"][a:b] if st["row_token"] is None else st["X"][st["row_token"][a:b].long()]
                Y[a:b] = _exact_product(x, st["codes"][e], st["scales"][e],
                                        None if st["zeros"] is None else st["zeros"][e], c["group"])
        if c["silu"]:
            half = c["N"] // 2
            Y = Y[:, :half] * torch.sigmoid(Y[:, :half]) * Y[:, half:]
        return Y
    if kind == "weights":
        # group by group; a code is the nearest multiple of the scale, found by comparing with the midpoints
        N, K = c["N"], c["K"]
        t = _TYPES[c["s"]]
        What = torch.empty((N, K), dtype=torch.float64, device="cuda")
        S, Z = [], []
        for k0 in range(0, K, c["group"]):
            w = st["W"][:, k0:k0 + c["group"]].double()
            if c["asym"]:
                lo = torch.minimum(w.min(1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
                hi = torch.maximum(w.max(1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
                s = ((hi - lo) / 15).clamp(max=torch.finfo(t).max).float().to(t).double()
                z = torch.where(s == 0, 0.0, _nearest(-lo[:, None], s[:, None])[:, 0].clamp(0, 15))
            else:
                s = (w.abs().max(1).values / 7).clamp(max=torch.finfo(t).max).float().to(t).double()
                z = torch.full_like(s, 8.0)
            n = _nearest(w, s[:, None])
            n = torch.minimum(torch.maximum(n, -z[:, None]), 15 - z[:, None])
            What[:, k0:k0 + c["group"]] = n * s[:, None]
            S.append(s)
            Z.append(z)
        out = (What, torch.stack(S, 1))
        return (*out, torch.stack(Z, 1).to(torch.uint8)) if c["asym"] else out
    T, k, D, R = c["T"], c["k"], c["D"], st["R"]
    rows = st["row_of"].tolist()
    flat = torch.tensor([f for f in range(T * k) if rows[f] >= 0], dtype=torch.int64, device="cuda")
    row = st["row_of"][flat].long()
    tok = flat // k
    w = torch.ones(R, dtype=torch.float64, device="cuda")
    if c["weighted"]:
        w = st["weights"].double().reshape(-1)[flat]
    if kind == "permute" and not c["back"]:
        out = torch.empty((R, D), dtype=torch.float64, device="cuda")
        out[row] = st["X"].double()[tok] * w[:, None]
        return out
    if kind == "unpermute" and c["back"]:
        dYp = torch.empty((R, D), dtype=torch.float64, device="cuda")
        dYp[row] = st["dout"].double()[tok] * w[:, None]
        return (dYp, _dots(st["dout"], st["Yp"], tok, row, flat, T, k)) if c["weighted"] else dYp
    src = st["dXp"] if kind == "permute" else st["Yp"]
    out = torch.zeros((T, D), dtype=torch.float64, device="cuda")
    out.index_add_(0, tok, src.double()[row] * w[:, None])
    if kind == "permute" and c["weighted"]:
        return out, _dots(st["X"], src, tok, row, flat, T, k)
    return out


def _nearest(w, s):
    """The whole number nearest to w / s, halves to the even one; 0 where s is 0."""
    n = torch.zeros_like(w)
    for i in range(1, 17):       # quotients of a group lie within its sixteen steps; beyond them the code clamps
        border = s * (i - 0.5)
        over = (w > border) if i % 2 else (w >= border)
        under = (w < -border) if i % 2 else (w <= -border)
        n = n + over.double() - under.double()
    return torch.where(s == 0, 0.0, n)


def _dots(A, B, tok, row, flat, T, k):
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    for i in range(0, flat.numel(), 4096):
        dw[flat[i:i + 4096]] = (A[tok[i:i + 4096]].double() * B[row[i:i + 4096]].double()).sum(1)
    return dw.view(T, k)
