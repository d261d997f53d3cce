"""Refusals of the integer 4-bit calls and of the token permutation, on the host and without a GPU."""
import ctypes
import os

import pytest
import torch

import structured_sparse_nvfp4_amd as ssn

pytestmark = pytest.mark.skipif(not os.path.exists(ssn.LIB_PATH), reason="library not built")

P, N0 = ctypes.c_void_p(0x1000), None


def at(a):
    return ctypes.c_void_p(a)


def _call(name, base, **change):
    args = dict(base)
    args.update(change)
    st = getattr(ssn.lib(), name)(*args.values())
    return st, ssn.lib().ssn_last_error()


QUANT = dict(W=P, w=0, N=4, K=64, group=32, s=1, codes=P, scales=P, zeros=P, stream=N0)
DEQUANT = dict(codes=P, scales=P, s=1, zeros=P, N=4, K=64, group=32, out=P, o=0, stream=N0)
GEMV = dict(X=P, x=1, M=2, N=4, K=64, codes=P, scales=P, s=1, zeros=P, group=32, Y=P, y=0, algo=0, used=N0, stream=N0)
GROUPED = dict(X=P, x=1, x_rows=8, row_token=P, offsets=P, E=4, R=8, N=32, K=64, codes=P, scales=P, s=1, zeros=P,
               group=32, epi=0, Y=P, y=0, algo=0, used=N0, stream=N0)
CASES = [
    ("int4_quantize", QUANT, dict(K=48), ssn.SSN_E_SHAPE), ("int4_quantize", QUANT, dict(N=-1), ssn.SSN_E_SHAPE),
    ("int4_quantize", QUANT, dict(group=0), ssn.SSN_E_RANGE), ("int4_quantize", QUANT, dict(group=-32), ssn.SSN_E_RANGE),
    ("int4_quantize", QUANT, dict(group=48), ssn.SSN_E_RANGE), ("int4_quantize", QUANT, dict(w=3), ssn.SSN_E_DTYPE),
    ("int4_quantize", QUANT, dict(s=0), ssn.SSN_E_DTYPE), ("int4_quantize", QUANT, dict(W=N0), ssn.SSN_E_NULL),
    ("int4_quantize", QUANT, dict(scales=N0), ssn.SSN_E_NULL), ("int4_quantize", QUANT, dict(codes=N0), ssn.SSN_E_NULL),
    ("int4_quantize", QUANT, dict(codes=at(0x1008)), ssn.SSN_E_ALIGN),
    ("int4_quantize", QUANT, dict(scales=at(0x1001)), ssn.SSN_E_ALIGN),
    ("int4_dequantize", DEQUANT, dict(K=16), ssn.SSN_E_SHAPE), ("int4_dequantize", DEQUANT, dict(o=9), ssn.SSN_E_DTYPE),
    ("int4_dequantize", DEQUANT, dict(s=0), ssn.SSN_E_DTYPE), ("int4_dequantize", DEQUANT, dict(group=31), ssn.SSN_E_RANGE),
    ("int4_dequantize", DEQUANT, dict(out=N0), ssn.SSN_E_NULL),
    ("int4_dequantize", DEQUANT, dict(scales=at(0x1003)), ssn.SSN_E_ALIGN),
    ("gemv_int4", GEMV, dict(K=40), ssn.SSN_E_SHAPE), ("gemv_int4", GEMV, dict(K=0), ssn.SSN_E_SHAPE),
    ("gemv_int4", GEMV, dict(M=-1), ssn.SSN_E_SHAPE), ("gemv_int4", GEMV, dict(M=1 << 31), ssn.SSN_E_SHAPE),
    ("gemv_int4", GEMV, dict(N=1 << 31), ssn.SSN_E_SHAPE), ("gemv_int4", GEMV, dict(group=33), ssn.SSN_E_RANGE),
    ("gemv_int4", GEMV, dict(x=0), ssn.SSN_E_DTYPE), ("gemv_int4", GEMV, dict(s=0), ssn.SSN_E_DTYPE),
    ("gemv_int4", GEMV, dict(y=5), ssn.SSN_E_DTYPE), ("gemv_int4", GEMV, dict(algo=ssn.ALGO_STREAM), ssn.SSN_E_ALGO),
    ("gemv_int4", GEMV, dict(X=N0), ssn.SSN_E_NULL), ("gemv_int4", GEMV, dict(Y=N0), ssn.SSN_E_NULL),
    ("gemv_int4", GEMV, dict(scales=N0), ssn.SSN_E_NULL), ("gemv_int4", GEMV, dict(X=at(0x1002)), ssn.SSN_E_ALIGN),
    ("gemv_int4", GEMV, dict(N=1 << 30, K=1 << 30), ssn.SSN_E_SHAPE),
    ("gemv_int4", GEMV, dict(K=(1 << 20) + 32), ssn.SSN_E_SHAPE), ("gemv_int4", GEMV, dict(M=(1 << 24) + 1), ssn.SSN_E_SHAPE),
    ("moe_grouped_gemv_int4", GROUPED, dict(R=(1 << 24) + 1), ssn.SSN_E_SHAPE),
    ("moe_grouped_gemv_int4", GROUPED, dict(K=(1 << 20) + 32), ssn.SSN_E_SHAPE),
    ("moe_grouped_gemv_int4", GROUPED, dict(E=0), ssn.SSN_E_RANGE),
    ("moe_grouped_gemv_int4", GROUPED, dict(E=4096), ssn.SSN_E_RANGE),
    ("moe_grouped_gemv_int4", GROUPED, dict(epi=2), ssn.SSN_E_RANGE),
    ("moe_grouped_gemv_int4", GROUPED, dict(epi=1, N=33), ssn.SSN_E_SHAPE),
    ("moe_grouped_gemv_int4", GROUPED, dict(algo=ssn.ALGO_MFMA), ssn.SSN_E_ALGO),
    ("moe_grouped_gemv_int4", GROUPED, dict(x_rows=0), ssn.SSN_E_SHAPE),
    ("moe_grouped_gemv_int4", GROUPED, dict(R=-1), ssn.SSN_E_SHAPE),
    ("moe_grouped_gemv_int4", GROUPED, dict(offsets=N0), ssn.SSN_E_NULL),
    ("moe_grouped_gemv_int4", GROUPED, dict(offsets=at(0x1002)), ssn.SSN_E_ALIGN),
    ("moe_grouped_gemv_int4", GROUPED, dict(row_token=at(0x1001)), ssn.SSN_E_ALIGN),
]


@pytest.mark.parametrize("name,base,change,want", CASES, ids=lambda v: v if isinstance(v, str) else None)
def test_int4_refusals(name, base, change, want):
    st, msg = _call(name, base, **change)
    assert st == want and name.encode() in msg


def test_int4_empty_problems_launch_nothing():
    used = ctypes.c_int(-1)
    assert _call("int4_quantize", QUANT, N=0, W=N0, codes=N0, scales=N0)[0] == ssn.SSN_OK
    assert _call("int4_dequantize", DEQUANT, K=0, out=N0)[0] == ssn.SSN_OK
    assert _call("gemv_int4", GEMV, M=0, X=N0, Y=N0, used=ctypes.byref(used))[0] == ssn.SSN_OK
    assert used.value == ssn.ALGO_MFMA
    assert _call("gemv_int4", GEMV, N=0, K=0, codes=N0)[0] == ssn.SSN_OK
    assert _call("moe_grouped_gemv_int4", GROUPED, R=0, x_rows=0, X=N0, offsets=N0, used=ctypes.byref(used))[0] == ssn.SSN_OK
    assert used.value == ssn.ALGO_STREAM


PERMUTE = dict(X=P, t=1, T=4, k=2, D=16, row_of=P, w=P, R=8, Xp=P, stream=N0)
PERMUTE_B = dict(dXp=P, t=1, R=8, row_of=P, w=P, T=4, k=2, D=16, X=P, dX=P, dw=P, stream=N0)
UNPERMUTE = dict(Yp=P, t=1, R=8, row_of=P, w=P, T=4, k=2, D=16, out=P, o=0, stream=N0)
UNPERMUTE_B = dict(dout=P, o=0, T=4, k=2, D=16, row_of=P, w=P, R=8, Yp=P, dYp=P, t=1, dw=P, stream=N0)
ALL = [("moe_permute", PERMUTE), ("moe_permute_backward", PERMUTE_B), ("moe_unpermute", UNPERMUTE),
       ("moe_unpermute_backward", UNPERMUTE_B)]


@pytest.mark.parametrize("name,base", ALL, ids=lambda v: v if isinstance(v, str) else None)
def test_permutation_refusals(name, base):
    for change, want in ((dict(k=0), ssn.SSN_E_RANGE), (dict(k=65), ssn.SSN_E_RANGE), (dict(T=-1), ssn.SSN_E_SHAPE),
                         (dict(D=-1), ssn.SSN_E_SHAPE), (dict(R=-1), ssn.SSN_E_SHAPE), (dict(R=1 << 31), ssn.SSN_E_SHAPE),
                         (dict(T=1 << 30, k=2), ssn.SSN_E_SHAPE), (dict(t=4), ssn.SSN_E_DTYPE),
                         (dict(row_of=N0), ssn.SSN_E_NULL), (dict(row_of=at(0x1002)), ssn.SSN_E_ALIGN),
                         (dict(w=at(0x1002)), ssn.SSN_E_ALIGN)):
        st, msg = _call(name, base, **change)
        assert st == want and name.encode() in msg, change
    for arg in base:
        if base[arg] is P and arg not in ("w", "dw", "row_of"):
            assert _call(name, base, **{arg: N0})[0] == ssn.SSN_E_NULL, arg
            assert _call(name, base, **{arg: at(0x1008)})[0] == ssn.SSN_E_ALIGN, arg
    if "dw" in base:
        assert _call(name, base, dw=at(0x1002))[0] == ssn.SSN_E_ALIGN
    if "o" in base:
        assert _call(name, base, o=ssn.SSN_F16)[0] == ssn.SSN_E_DTYPE      # neither f32 nor the rows' bf16
    assert _call(name, base, T=0)[0] == ssn.SSN_OK


def test_permutation_empty_problems_launch_nothing():
    assert _call("moe_permute", PERMUTE, R=0, Xp=N0)[0] == ssn.SSN_OK
    assert _call("moe_permute", PERMUTE, D=0, X=N0)[0] == ssn.SSN_OK
    assert _call("moe_unpermute", UNPERMUTE, D=0, out=N0)[0] == ssn.SSN_OK
    assert _call("moe_permute_backward", PERMUTE_B, D=0, dw=N0)[0] == ssn.SSN_OK
    assert _call("moe_unpermute_backward", UNPERMUTE_B, R=0, dw=N0)[0] == ssn.SSN_OK


@pytest.mark.parametrize("name,args", [("moe_permute_backward", ("X", "dX")), ("moe_unpermute", ("out",)),
                                       ("moe_unpermute_backward", ("dout",))])
def test_token_side_is_checked_without_rows(name, args):
    """R = 0: the token side still has T rows, and what launches checks it first."""
    for arg in args:
        assert _call(name, dict(ALL)[name], R=0, **{arg: N0})[0] == ssn.SSN_E_NULL, arg
        assert _call(name, dict(ALL)[name], R=0, **{arg: at(0x1008)})[0] == ssn.SSN_E_ALIGN, arg


def test_half_type_is_still_refused_by_the_other_calls():
    L = ssn.lib()
    assert L.gemm_nvfp4_dense(P, 2, 4, 64, P, P, P, P, ssn.SSN_F16, 0, N0, N0) == ssn.SSN_E_DTYPE
    assert L.moe_combine(P, ssn.SSN_F16, 4, P, P, 2, 2, 16, P, N0) == ssn.SSN_E_DTYPE


def test_binding_refusals():
    """What the binding refuses before it looks for a device; tensors on the host are refused as such."""
    W, c = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8)
    s, x = torch.zeros(4, 2, dtype=torch.bfloat16), torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        ssn.int4_quantize(W, group=32)
    with pytest.raises(ValueError, match="dimensions"):
        ssn.int4_quantize(W[0])
    with pytest.raises(ValueError, match="dimensions"):
        ssn.gemv_int4(x[0], c, s, group=32)
    with pytest.raises(TypeError, match="Tensor"):
        ssn.gemv_int4([1.0], c, s)
    with pytest.raises(TypeError, match="X must be one of"):
        ssn.gemv_int4(W, c, s, group=32)
    with pytest.raises(TypeError, match="scales must be one of"):
        ssn.gemv_int4(x, c, s.float(), group=32)
    for group in (0, 48, -32, 32.0, True):
        with pytest.raises(ValueError, match="multiple of 32"):
            ssn.int4_dequantize(c, s, group=group)
    with pytest.raises(ValueError, match="device"):
        ssn.moe_permute(x, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        ssn.moe_unpermute(x[0], torch.zeros(4, dtype=torch.int32), 2)
    for group in (1 << 62, (1 << 64) + 32):               # beyond the 64 bits of the call
        with pytest.raises(ValueError, match="too large"):
            ssn.gemv_int4(x, c, s[:, :1].contiguous(), group=group)
