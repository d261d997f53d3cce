"""Refusals of the 4-bit cache's calls, on the host and without a GPU."""
import ctypes
import os

import pytest
import torch

import structured_sparse_nvfp4_amd as ssn

pytestmark = pytest.mark.skipif(not os.path.exists(ssn.LIB_PATH), reason="library not built")

P, N0 = ctypes.c_void_p(0x1000), None
BIG = 1 << 40


def at(a):
    return ctypes.c_void_p(a)


def _call(name, base, **change):
    args = dict(base)
    args.update(change)
    st = getattr(ssn.lib(), name)(*args.values())
    return st, ssn.lib().ssn_last_error()


CACHE = dict(kc=P, ks=P, vc=P, vs=P, kt=P, vt=P, pages=4, page=16, Hkv=2, D=64)
APPEND = dict(K=P, V=P, dt=1, T=3, kts=128, khs=64, vts=128, vhs=64, slots=P, **CACHE, bad=N0, stream=N0)
READ = dict(slots=P, T=3, **CACHE, K=P, V=P, dt=1, stream=N0)
ATTN = dict(Q=P, qt=1, Tq=4, Hq=4, qts=256, qhs=64, **CACHE, table=P, B=2, blocks=4, lens=P, offs=N0, max_q=2, max_kv=64,
            scale=0.125, causal=1, window=0, out=P, ot=1, lse=N0, algo=0, used=N0, ws=N0, wsb=0, stream=N0)
SHARED = [
    (dict(D=48), ssn.SSN_E_SHAPE), (dict(D=0), ssn.SSN_E_SHAPE), (dict(D=288), ssn.SSN_E_SHAPE), (dict(D=-32), ssn.SSN_E_SHAPE),
    (dict(page=8), ssn.SSN_E_SHAPE), (dict(page=24), ssn.SSN_E_SHAPE), (dict(page=-16), ssn.SSN_E_SHAPE),
    (dict(page=(1 << 20) + 16), ssn.SSN_E_SHAPE), (dict(pages=0), ssn.SSN_E_SHAPE), (dict(pages=1 << 31), ssn.SSN_E_SHAPE),
    (dict(pages=1 << 25, page=1 << 16), ssn.SSN_E_SHAPE),
    (dict(Hkv=0), ssn.SSN_E_RANGE), (dict(Hkv=4097), ssn.SSN_E_RANGE), (dict(kc=N0), ssn.SSN_E_NULL),
    (dict(ks=N0), ssn.SSN_E_NULL), (dict(vc=N0), ssn.SSN_E_NULL), (dict(vs=N0), ssn.SSN_E_NULL), (dict(kt=N0), ssn.SSN_E_NULL),
    (dict(vt=N0), ssn.SSN_E_NULL), (dict(kc=at(0x1008)), ssn.SSN_E_ALIGN), (dict(vs=at(0x1004)), ssn.SSN_E_ALIGN),
    (dict(kt=at(0x1002)), ssn.SSN_E_ALIGN),
]
CASES = [(n, b, c, s) for n, b in (("kv_nvfp4_append", APPEND), ("kv_nvfp4_read", READ), ("attn_kv_nvfp4", ATTN))
         for c, s in SHARED] + [
    ("kv_nvfp4_append", APPEND, dict(T=-1), ssn.SSN_E_SHAPE), ("kv_nvfp4_append", APPEND, dict(T=(1 << 26) + 1), ssn.SSN_E_SHAPE),
    ("kv_nvfp4_append", APPEND, dict(dt=3), ssn.SSN_E_DTYPE), ("kv_nvfp4_append", APPEND, dict(K=N0), ssn.SSN_E_NULL),
    ("kv_nvfp4_append", APPEND, dict(V=at(0x1002)), ssn.SSN_E_ALIGN), ("kv_nvfp4_append", APPEND, dict(slots=N0), ssn.SSN_E_NULL),
    ("kv_nvfp4_append", APPEND, dict(slots=at(0x1004)), ssn.SSN_E_ALIGN), ("kv_nvfp4_append", APPEND, dict(bad=at(0x1004)), ssn.SSN_E_ALIGN),
    ("kv_nvfp4_append", APPEND, dict(kts=100), ssn.SSN_E_ALIGN), ("kv_nvfp4_append", APPEND, dict(vhs=4, dt=1), ssn.SSN_E_ALIGN),
    ("kv_nvfp4_append", APPEND, dict(vhs=2, dt=0), ssn.SSN_E_ALIGN), ("kv_nvfp4_append", APPEND, dict(khs=-64), ssn.SSN_E_SHAPE),
    ("kv_nvfp4_append", APPEND, dict(vts=BIG + 8), ssn.SSN_E_SHAPE),
    ("kv_nvfp4_read", READ, dict(T=-1), ssn.SSN_E_SHAPE), ("kv_nvfp4_read", READ, dict(dt=9), ssn.SSN_E_DTYPE),
    ("kv_nvfp4_read", READ, dict(T=(1 << 26) + 1), ssn.SSN_E_SHAPE), ("kv_nvfp4_read", READ, dict(K=N0), ssn.SSN_E_NULL),
    ("kv_nvfp4_read", READ, dict(V=at(0x1008)), ssn.SSN_E_ALIGN), ("kv_nvfp4_read", READ, dict(slots=N0), ssn.SSN_E_NULL),
    ("attn_kv_nvfp4", ATTN, dict(qt=0), ssn.SSN_E_DTYPE), ("attn_kv_nvfp4", ATTN, dict(ot=2), ssn.SSN_E_DTYPE),
    ("attn_kv_nvfp4", ATTN, dict(ot=7), ssn.SSN_E_DTYPE), ("attn_kv_nvfp4", ATTN, dict(Hq=3), ssn.SSN_E_RANGE),
    ("attn_kv_nvfp4", ATTN, dict(Hq=0), ssn.SSN_E_RANGE), ("attn_kv_nvfp4", ATTN, dict(Hq=1), ssn.SSN_E_RANGE),
    ("attn_kv_nvfp4", ATTN, dict(Tq=5), ssn.SSN_E_SHAPE), ("attn_kv_nvfp4", ATTN, dict(Tq=-2), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(B=-1), ssn.SSN_E_SHAPE), ("attn_kv_nvfp4", ATTN, dict(B=(1 << 20) + 1), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(max_q=-1), ssn.SSN_E_SHAPE), ("attn_kv_nvfp4", ATTN, dict(max_q=1 << 30), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(max_kv=65), ssn.SSN_E_SHAPE), ("attn_kv_nvfp4", ATTN, dict(max_kv=-1), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(max_kv=(1 << 27) + 1, blocks=1 << 30), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(blocks=-1), ssn.SSN_E_SHAPE), ("attn_kv_nvfp4", ATTN, dict(window=-1), ssn.SSN_E_RANGE),
    ("attn_kv_nvfp4", ATTN, dict(window=1 << 31), ssn.SSN_E_RANGE), ("attn_kv_nvfp4", ATTN, dict(window=5, causal=0), ssn.SSN_E_RANGE),
    ("attn_kv_nvfp4", ATTN, dict(scale=float("nan")), ssn.SSN_E_RANGE), ("attn_kv_nvfp4", ATTN, dict(scale=float("inf")), ssn.SSN_E_RANGE),
    ("attn_kv_nvfp4", ATTN, dict(algo=ssn.ALGO_VALU), ssn.SSN_E_ALGO), ("attn_kv_nvfp4", ATTN, dict(algo=99), ssn.SSN_E_ALGO),
    ("attn_kv_nvfp4", ATTN, dict(qts=100), ssn.SSN_E_ALIGN), ("attn_kv_nvfp4", ATTN, dict(qhs=-64), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(Q=N0), ssn.SSN_E_NULL), ("attn_kv_nvfp4", ATTN, dict(out=at(0x1008)), ssn.SSN_E_ALIGN),
    ("attn_kv_nvfp4", ATTN, dict(lens=N0), ssn.SSN_E_NULL), ("attn_kv_nvfp4", ATTN, dict(lens=at(0x1002)), ssn.SSN_E_ALIGN),
    ("attn_kv_nvfp4", ATTN, dict(table=N0), ssn.SSN_E_NULL), ("attn_kv_nvfp4", ATTN, dict(offs=at(0x1001)), ssn.SSN_E_ALIGN),
    ("attn_kv_nvfp4", ATTN, dict(lse=at(0x1002)), ssn.SSN_E_ALIGN),
    # a long sequence needs a workspace
    ("attn_kv_nvfp4", ATTN, dict(blocks=1 << 13, max_kv=1 << 17), ssn.SSN_E_NULL),
    ("attn_kv_nvfp4", ATTN, dict(blocks=1 << 13, max_kv=1 << 17, ws=P, wsb=64), ssn.SSN_E_RANGE),
    ("attn_kv_nvfp4", ATTN, dict(blocks=1 << 13, max_kv=1 << 17, ws=at(0x1004), wsb=1 << 30), ssn.SSN_E_ALIGN),
    ("attn_kv_nvfp4", ATTN, dict(B=65535, Hkv=4096, Hq=4096, Tq=65535, max_q=1), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(B=65536, Tq=65536, max_q=1), ssn.SSN_E_SHAPE),
    ("attn_kv_nvfp4", ATTN, dict(B=1, Hkv=1, Hq=1, Tq=1 << 24, max_q=1 << 24, algo=ssn.ALGO_STREAM), ssn.SSN_E_SHAPE),
]


@pytest.mark.parametrize("name,base,change,status", CASES, ids=[f"{c[0]}-{i}" for i, c in enumerate(CASES)])
def test_refused_before_any_launch(name, base, change, status):
    st, msg = _call(name, base, **change)
    assert st == status, (st, msg)
    assert msg.startswith(name.encode())


def test_empty_calls():
    assert _call("kv_nvfp4_append", APPEND, T=0, K=N0, V=N0, slots=N0)[0] == ssn.SSN_OK
    assert _call("kv_nvfp4_read", READ, T=0, K=N0, V=N0, slots=N0)[0] == ssn.SSN_OK
    for change in (dict(Tq=0), dict(B=0, Tq=4), dict(max_q=0)):
        used = ctypes.c_int(-1)
        st, msg = _call("attn_kv_nvfp4", ATTN, Q=N0, out=N0, table=N0, lens=N0, used=ctypes.byref(used), **change)
        assert st == ssn.SSN_OK and used.value in (ssn.ALGO_STREAM, ssn.ALGO_MFMA), msg


def test_workspace_sizes():
    f = ssn.lib().attn_kv_nvfp4_workspace_bytes
    assert f(2, 4, 3, 64, 1, 100) == -1 and f(2, 4, 2, 40, 1, 100) == -1 and f(-1, 4, 2, 64, 1, 100) == -1
    assert f(2, 4, 2, 64, -1, 100) == -1 and f(2, 4, 2, 64, 1, (1 << 27) + 1) == -1
    assert f(0, 4, 2, 64, 1, 100) == 0 and f(2, 4, 2, 64, 0, 100) == 0 and f(2, 4, 2, 64, 1, 0) == 0
    assert f(2, 4, 2, 64, 1, 64) == 0
    assert f(1, 64, 8, 128, 1, 131072) > 0
    assert f(65535, 4096, 4096, 256, 1 << 20, 1 << 27) == 0 and f(65536, 4, 2, 64, 1, 100) == -1


def test_the_binding_refuses():
    """What the binding can see without a device."""
    c = ssn.KvNvfp4(*(torch.zeros(s, dtype=torch.uint8) for s in ((2, 2, 16, 32), (2, 2, 16, 4), (2, 2, 16, 32), (2, 2, 4, 16))),
                    torch.ones(2), torch.ones(2))
    K, slots = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    for bad, err in ((dict(cache=c._replace(v_scales=c.k_scales)), ValueError), (dict(cache=c._replace(k_codes=c.k_codes.float())), TypeError),
                     (dict(cache=c._replace(k_tensor_scale=torch.ones(3))), ValueError), (dict(K=K[:, :1]), ValueError),
                     (dict(V=K.half()), TypeError), (dict(K=K.double(), V=K.double()), TypeError), (dict(slots=slots.int()), TypeError),
                     (dict(slots=slots[:2]), ValueError), (dict(K=K.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                     (dict(K="K"), TypeError), (dict(cache=c._replace(v_codes=None)), TypeError), (dict(cache=c._replace(k_codes=c.k_codes[:, :, ::2])), ValueError)):
        with pytest.raises(err):
            ssn.kv_nvfp4_append(**{**dict(K=K, V=K, slots=slots, cache=c), **bad})
    with pytest.raises(ValueError, match="device tensors"):
        ssn.kv_nvfp4_append(K, K, slots, c)
    for bad, err in ((dict(slots=slots.int()), TypeError), (dict(slots=slots[None]), ValueError), (dict(out_dtype=torch.int8), TypeError),
                     (dict(K=torch.zeros(2, 2, 64)), ValueError), (dict(V=torch.zeros(3, 2, 64)), TypeError)):
        with pytest.raises(err):
            ssn.kv_nvfp4_read(**{**dict(slots=slots, cache=c), **bad})
    with pytest.raises(ValueError, match="device tensors"):
        ssn.kv_nvfp4_read(slots, c)
    Q, table, lens = torch.zeros(2, 4, 64).half(), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = dict(Q=Q, cache=c, block_table=table, seq_lens=lens)
    for bad, err in ((dict(Q=Q.float()), TypeError), (dict(Q=Q[:, :, :32]), ValueError), (dict(block_table=table.long()), TypeError),
                     (dict(seq_lens=lens[:1]), ValueError), (dict(q_offsets=lens), ValueError), (dict(out_dtype=torch.bfloat16), TypeError),
                     (dict(out=torch.zeros(2, 4, 32).half()), ValueError), (dict(lse=torch.zeros(2, 4).half()), TypeError),
                     (dict(Q=Q[:, :3]), ssn.SsnError), (dict(max_kv=1 << 28), ssn.SsnError), (dict(max_q=-1), ssn.SsnError),
                     (dict(block_table=table[0]), ValueError), (dict(workspace=lens), TypeError)):
        with pytest.raises(err):
            ssn.attn_kv_nvfp4(**{**good, **bad})
    with pytest.raises(ValueError, match="device tensors"):
        ssn.attn_kv_nvfp4(**good)
