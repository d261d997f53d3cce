"""Python binding of ``libssnvfp4.so`` — NVFP4 / 2:4 weight-quantised GEMM for MI355X (gfx950).

Argument marshalling only: every step runs in the library's HIP kernels. PyTorch supplies
device memory and the current stream. The functions have the names of the C entry points
declared in ``include/ssnvfp4.h``; outputs are allocated here with torch when not given.
If the shared library is missing, every call raises (there is no fallback).

No call records itself for torch's automatic differentiation: results never require a gradient, whatever the
inputs do. ``moe_permute`` and ``moe_unpermute`` have theirs as calls (``moe_permute_backward``,
``moe_unpermute_backward``), to be made by hand or from a ``torch.autograd.Function`` of the caller's.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssnvfp4.so")

SSN_OK, SSN_E_NULL, SSN_E_SHAPE, SSN_E_ALIGN, SSN_E_DTYPE, SSN_E_ALGO, SSN_E_HIP, SSN_E_RANGE = range(8)
SSN_F32, SSN_BF16, SSN_F16 = 0, 1, 2
ALGO_AUTO, ALGO_VALU, ALGO_MFMA, ALGO_SMFMAC, ALGO_GATHER, ALGO_DECOMPRESS_MFMA, ALGO_STREAM = 0, 1, 2, 3, 4, 5, 6
ALGO_NAMES = {ALGO_AUTO: "auto", ALGO_VALU: "valu", ALGO_MFMA: "mfma", ALGO_SMFMAC: "smfmac", ALGO_GATHER: "gather",
              ALGO_DECOMPRESS_MFMA: "decompress_mfma", ALGO_STREAM: "stream"}
EPI_NONE, EPI_SILU_GATE = 0, 1
MX_ROWS, MX_TILED = 0, 1
WLAYOUT_ROWS, WLAYOUT_KTILE64 = 0, 1
PROBE_BF16, PROBE_FP4 = 0, 1

_vp, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SIGS = {
    "ssn_last_error": ([], ctypes.c_char_p),
    "ssn_version": ([], _int),
    "nvfp4_quantize": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, _vp], _int),
    "nvfp4_dequantize": ([_vp, _vp, _vp, _i64, _i64, _vp, _int, _vp], _int),
    "nvfp4_sp24_produce": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _int),
    "sp24_prune": ([_vp, _int, _i64, _i64, _vp, _vp, _vp], _int),
    "sp24_check": ([_vp, _i64, _i64, _vp, _vp, _vp], _int),
    "sp24_compress": ([_vp, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "sp24_decompress": ([_vp, _vp, _i64, _i64, _vp, _vp], _int),
    "gemm_nvfp4_dense": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _int, _int, _vp, _vp], _int),
    "gemm_nvfp4_sp24": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _int, _int, _vp, _vp], _int),
    "moe_route_workspace_bytes": ([_i64, _int, _int], _i64),
    "moe_route": ([_vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "moe_grouped_gemm_nvfp4": ([_vp, _i64, _vp, _vp, _int, _i64, _i64, _i64, _int, _int, _vp, _vp, _vp, _vp,
                                _int, _vp, _int, _int, _vp, _vp], _int),
    "moe_pack_ktiles": ([_vp, _i64, _i64, _i64, _i64, _vp, _vp], _int),
    "moe_combine": ([_vp, _int, _i64, _vp, _vp, _i64, _int, _i64, _vp, _vp], _int),
    "moe_ffn_workspace_bytes": ([_i64, _int, _int, _i64, _i64], _i64),
    "moe_nvfp4_ffn": ([_vp, _i64, _i64, _vp, _vp, _int, _int, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp,
                       _vp, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "mxfp4_tiled_bytes": ([_i64, _i64, _vp], _i64),
    "mxfp4_quantize": ([_vp, _int, _i64, _i64, _int, _vp, _vp, _vp], _int),
    "gemm_mxfp4": ([_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _int, _int, _vp, _vp], _int),
    "moe_nvfp4_ffn_noalloc": ([_vp, _i64, _i64, _vp, _vp, _int, _int, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp,
                               _vp, _vp, _vp, _vp, _vp, _vp], _int),
    "int4_quantize": ([_vp, _int, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp], _int),
    "int4_dequantize": ([_vp, _vp, _int, _vp, _i64, _i64, _i64, _vp, _int, _vp], _int),
    "gemv_int4": ([_vp, _int, _i64, _i64, _i64, _vp, _vp, _int, _vp, _i64, _vp, _int, _int, _vp, _vp], _int),
    "moe_grouped_gemv_int4": ([_vp, _int, _i64, _vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, _int, _vp, _i64, _int,
                               _vp, _int, _int, _vp, _vp], _int),
    "moe_permute": ([_vp, _int, _i64, _int, _i64, _vp, _vp, _i64, _vp, _vp], _int),
    "moe_permute_backward": ([_vp, _int, _i64, _vp, _vp, _i64, _int, _i64, _vp, _vp, _vp, _vp], _int),
    "moe_unpermute": ([_vp, _int, _i64, _vp, _vp, _i64, _int, _i64, _vp, _int, _vp], _int),
    "moe_unpermute_backward": ([_vp, _int, _i64, _int, _i64, _vp, _vp, _i64, _vp, _vp, _int, _vp, _vp], _int),
    "kv_nvfp4_append": ([_vp, _vp, _int, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _int,
                         _int, _int, _vp, _vp], _int),
    "kv_nvfp4_read": ([_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _vp, _vp, _int, _vp], _int),
    "attn_kv_nvfp4": ([_vp, _int, _i64, _int, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _vp,
                       _i64, _i64, _vp, _vp, _i64, _i64, ctypes.c_float, _int, _i64, _vp, _int, _vp, _int, _vp, _vp,
                       _i64, _vp], _int),
    "attn_kv_nvfp4_workspace_bytes": ([_i64, _int, _int, _int, _i64, _i64], _i64),
    "mfma_probe_sink_floats": ([], _i64),
    "mfma_probe": ([_int, _int, _int, ctypes.c_uint32, _vp, _vp, _vp], _int),
}

_lib = None


class SsnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"[status {status}] {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python structured_sparse_nvfp4_amd/build.py` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def _check(status: int):
    if status != SSN_OK:
        raise SsnError(status, lib().ssn_last_error().decode())


class Prepared:
    """A call with its arguments already marshalled (tensors, sizes, stream): calling it issues
    the C entry point with no per-call Python work beyond the ctypes call itself. Used to keep the
    host ahead of the GPU when timing short kernels. The tensors must stay alive."""

    def __init__(self, fname, cargs, keep):
        self.f = getattr(lib(), fname)
        self.cargs = cargs
        self.keep = keep

    def __call__(self):
        st = self.f(*self.cargs)
        if st:
            _check(st)


def _run(fname, cargs, prepare, keep, result):
    if prepare:   # the prepared call holds its outputs too: they must outlive every later call
        return Prepared(fname, cargs, (keep, result)), result
    _check(getattr(lib(), fname)(*cargs))
    return result


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev=None):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, dtype, name, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _wdt(W):
    if W.dtype == torch.float32:
        return SSN_F32
    if W.dtype == torch.bfloat16:
        return SSN_BF16
    raise TypeError(f"weights must be float32 or bfloat16, got {W.dtype}")


def version() -> int:
    return lib().ssn_version()


def nvfp4_quantize(W, tensor_scale_in=None, codes=None, scales=None, tensor_scale_out=None, prepare=False):
    """NVFP4-quantise W [N, K] (f32 or bf16). Returns (codes u8 [N,K/2], scales u8 [N,K/16], s_t f32 [1])."""
    N, K = W.shape
    _need(W, W.dtype, "W")
    dev = W.device
    codes = codes if codes is not None else torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = scales if scales is not None else torch.empty((N, K // 16), dtype=torch.uint8, device=dev)
    ts = tensor_scale_out if tensor_scale_out is not None else torch.empty(1, dtype=torch.float32, device=dev)
    _need(codes, torch.uint8, "codes", (N, K // 2)); _need(scales, torch.uint8, "scales", (N, K // 16))
    _need(ts, torch.float32, "tensor_scale_out", (1,))
    if tensor_scale_in is not None:
        _need(tensor_scale_in, torch.float32, "tensor_scale_in", (1,))
    cargs = (_ptr(W), _wdt(W), N, K, _ptr(tensor_scale_in), _ptr(codes), _ptr(scales), _ptr(ts), _stream(dev))
    return _run("nvfp4_quantize", cargs, prepare, (W, tensor_scale_in), (codes, scales, ts))


def nvfp4_dequantize(codes, scales, tensor_scale, out_dtype=torch.float32, out=None):
    N, Kh = codes.shape
    K = 2 * Kh
    _need(codes, torch.uint8, "codes"); _need(scales, torch.uint8, "scales", (N, K // 16))
    _need(tensor_scale, torch.float32, "tensor_scale", (1,))
    out = out if out is not None else torch.empty((N, K), dtype=out_dtype, device=codes.device)
    dt = SSN_F32 if out.dtype == torch.float32 else SSN_BF16 if out.dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError("out must be float32 or bfloat16")
    _need(out, out.dtype, "out", (N, K))
    _check(lib().nvfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(tensor_scale), N, K, _ptr(out), dt,
                                  _stream(codes.device)))
    return out


def nvfp4_sp24_produce(W, tensor_scale_in=None, vals=None, meta=None, scales=None, tensor_scale_out=None,
                       codes=None, want_codes=False, bad_groups=None, prepare=False):
    """Prune -> quantise -> compress W [N, K] (f32 or bf16) in one pass, bit-identical to sp24_prune,
    nvfp4_quantize and sp24_compress in turn. Returns (vals u8 [N,K/4], meta u8 [N,K/8], scales u8
    [N,K/16], s_t f32 [1], bad_groups int64 [1] device, codes u8 [N,K/2] of the pruned tensor or None)."""
    N, K = W.shape
    _need(W, W.dtype, "W")
    dev = W.device
    u8 = dict(dtype=torch.uint8, device=dev)
    vals = vals if vals is not None else torch.empty((N, K // 4), **u8)
    meta = meta if meta is not None else torch.empty((N, K // 8), **u8)
    scales = scales if scales is not None else torch.empty((N, K // 16), **u8)
    ts = tensor_scale_out if tensor_scale_out is not None else torch.empty(1, dtype=torch.float32, device=dev)
    bad = bad_groups if bad_groups is not None else torch.empty(1, dtype=torch.int64, device=dev)
    if codes is None and want_codes:
        codes = torch.empty((N, K // 2), **u8)
    _need(vals, torch.uint8, "vals", (N, K // 4)); _need(meta, torch.uint8, "meta", (N, K // 8))
    _need(scales, torch.uint8, "scales", (N, K // 16)); _need(ts, torch.float32, "tensor_scale_out", (1,))
    _need(bad, torch.int64, "bad_groups", (1,))
    if codes is not None:
        _need(codes, torch.uint8, "codes", (N, K // 2))
    if tensor_scale_in is not None:
        _need(tensor_scale_in, torch.float32, "tensor_scale_in", (1,))
    cargs = (_ptr(W), _wdt(W), N, K, _ptr(tensor_scale_in), _ptr(vals), _ptr(meta), _ptr(scales), _ptr(ts),
             _ptr(codes), _ptr(bad), _stream(dev))
    return _run("nvfp4_sp24_produce", cargs, prepare, (W, tensor_scale_in), (vals, meta, scales, ts, bad, codes))


def sp24_prune(W, out=None, tensor_scale_out=None, prepare=False):
    """2:4 magnitude prune along K (keep the two largest |w| of every group of four). With
    tensor_scale_out (f32 [1]) it also receives s_t of W, which is s_t of the pruned tensor too."""
    N, K = W.shape
    _need(W, W.dtype, "W")
    out = out if out is not None else torch.empty_like(W)
    _need(out, W.dtype, "out", (N, K))
    if tensor_scale_out is not None:
        _need(tensor_scale_out, torch.float32, "tensor_scale_out", (1,))
    cargs = (_ptr(W), _wdt(W), N, K, _ptr(out), _ptr(tensor_scale_out), _stream(W.device))
    return _run("sp24_prune", cargs, prepare, (W, tensor_scale_out), out)


def sp24_check(codes, bad_groups=None, first_bad=None, prepare=False):
    """Per-group 2:4 check. Returns device int64 tensors (bad_groups [1], first_bad [1])."""
    N, Kh = codes.shape
    _need(codes, torch.uint8, "codes")
    dev = codes.device
    bad = bad_groups if bad_groups is not None else torch.empty(1, dtype=torch.int64, device=dev)
    first = first_bad if first_bad is not None else torch.empty(1, dtype=torch.int64, device=dev)
    cargs = (_ptr(codes), N, 2 * Kh, _ptr(bad), _ptr(first), _stream(dev))
    return _run("sp24_check", cargs, prepare, (codes,), (bad, first))


def sp24_compress(codes, vals=None, meta=None, bad_groups=None, raise_if_bad=False, prepare=False):
    """2:4 compression. Returns (vals u8 [N,K/4], meta u8 [N,K/8], bad_groups int64 [1] device)."""
    N, Kh = codes.shape
    K = 2 * Kh
    _need(codes, torch.uint8, "codes")
    dev = codes.device
    vals = vals if vals is not None else torch.empty((N, K // 4), dtype=torch.uint8, device=dev)
    meta = meta if meta is not None else torch.empty((N, K // 8), dtype=torch.uint8, device=dev)
    bad = bad_groups if bad_groups is not None else torch.empty(1, dtype=torch.int64, device=dev)
    _need(vals, torch.uint8, "vals", (N, K // 4)); _need(meta, torch.uint8, "meta", (N, K // 8))
    cargs = (_ptr(codes), N, K, _ptr(vals), _ptr(meta), _ptr(bad), _stream(dev))
    if prepare:
        return _run("sp24_compress", cargs, True, (codes,), (vals, meta, bad))
    _check(lib().sp24_compress(*cargs))
    if raise_if_bad:
        nb = int(bad.item())
        if nb:
            raise ValueError(f"sp24_compress: {nb} group(s) of four have fewer than two zeros")
    return vals, meta, bad


def sp24_decompress(vals, meta, codes=None):
    N, G = vals.shape
    K = 4 * G
    _need(vals, torch.uint8, "vals"); _need(meta, torch.uint8, "meta", (N, K // 8))
    codes = codes if codes is not None else torch.empty((N, K // 2), dtype=torch.uint8, device=vals.device)
    _need(codes, torch.uint8, "codes", (N, K // 2))
    _check(lib().sp24_decompress(_ptr(vals), _ptr(meta), N, K, _ptr(codes), _stream(vals.device)))
    return codes


def _gemm_out(X, N, y_dtype, Y):
    M = X.shape[0]
    Y = Y if Y is not None else torch.empty((M, N), dtype=y_dtype, device=X.device)
    dt = SSN_F32 if Y.dtype == torch.float32 else SSN_BF16 if Y.dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError("Y must be float32 or bfloat16")
    _need(Y, Y.dtype, "Y", (M, N))
    return Y, dt


def gemm_nvfp4_dense(X, codes, scales, tensor_scale, y_dtype=torch.float32, algo=ALGO_AUTO, Y=None, prepare=False):
    """Y = X . W_hat^T for dense NVFP4 weights. Returns (Y, algorithm that ran)."""
    M, K = X.shape
    N = codes.shape[0]
    _need(X, torch.bfloat16, "X"); _need(codes, torch.uint8, "codes", (N, K // 2))
    _need(scales, torch.uint8, "scales", (N, K // 16)); _need(tensor_scale, torch.float32, "tensor_scale", (1,))
    Y, dt = _gemm_out(X, N, y_dtype, Y)
    used = ctypes.c_int(-1)
    cargs = (_ptr(X), M, N, K, _ptr(codes), _ptr(scales), _ptr(tensor_scale), _ptr(Y), dt, algo,
             ctypes.byref(used), _stream(X.device))
    if prepare:
        return Prepared("gemm_nvfp4_dense", cargs, (X, codes, scales, tensor_scale, used, Y)), (Y, used)
    _check(lib().gemm_nvfp4_dense(*cargs))
    return Y, used.value


def gemm_nvfp4_sp24(X, vals, meta, scales, tensor_scale, y_dtype=torch.float32, algo=ALGO_AUTO, Y=None,
                    prepare=False):
    """Y = X . W_hat^T from 2:4-compressed NVFP4 weights. Returns (Y, algorithm that ran)."""
    M, K = X.shape
    N = vals.shape[0]
    _need(X, torch.bfloat16, "X"); _need(vals, torch.uint8, "vals", (N, K // 4))
    _need(meta, torch.uint8, "meta", (N, K // 8)); _need(scales, torch.uint8, "scales", (N, K // 16))
    _need(tensor_scale, torch.float32, "tensor_scale", (1,))
    Y, dt = _gemm_out(X, N, y_dtype, Y)
    used = ctypes.c_int(-1)
    cargs = (_ptr(X), M, N, K, _ptr(vals), _ptr(meta), _ptr(scales), _ptr(tensor_scale), _ptr(Y), dt, algo,
             ctypes.byref(used), _stream(X.device))
    if prepare:
        return Prepared("gemm_nvfp4_sp24", cargs, (X, vals, meta, scales, tensor_scale, used, Y)), (Y, used)
    _check(lib().gemm_nvfp4_sp24(*cargs))
    return Y, used.value


# ------------------------------------------------------------------------------------------------
# grouped-expert (MoE) path


def moe_route(topk_ids, E, prepare=False):
    """Routing bookkeeping for topk_ids int32 [T, k]. Returns device tensors
    (expert_offsets [E+1], row_token [T*k], row_slot [T*k], row_of [T*k], bad_ids [1])."""
    T, k = topk_ids.shape
    _need(topk_ids, torch.int32, "topk_ids")
    dev = topk_ids.device
    F = T * k
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_token = torch.empty(max(F, 1), dtype=torch.int32, device=dev)[:F]
    row_slot = torch.empty(max(F, 1), dtype=torch.int32, device=dev)[:F]
    row_of = torch.empty(max(F, 1), dtype=torch.int32, device=dev)[:F]
    bad = torch.empty(1, dtype=torch.int64, device=dev)
    nws = lib().moe_route_workspace_bytes(T, k, E)
    if nws < 0:
        _check(lib().moe_route(None, T, k, E, None, None, None, None, None, None, 0, None))
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    cargs = (_ptr(topk_ids), T, k, E, _ptr(offsets), _ptr(row_token), _ptr(row_slot), _ptr(row_of), _ptr(bad),
             _ptr(ws), nws, _stream(dev))
    return _run("moe_route", cargs, prepare, (topk_ids, ws), (offsets, row_token, row_slot, row_of, bad))


def moe_grouped_gemm_nvfp4(X, row_token, expert_offsets, R, w_main, w_scales, tensor_scales, w_meta=None,
                           epilogue=EPI_NONE, y_dtype=torch.float32, algo=ALGO_AUTO, Y=None, prepare=False,
                           w_layout=WLAYOUT_ROWS):
    """Every expert's product in one launch. X bf16 [x_rows, K]; row_token int32 [R] or None
    (identity); expert_offsets int32 [E+1]; dense weights w_main [E, N, K/2] (w_meta None) or
    2:4 w_main [E, N, K/4] with w_meta [E, N, K/8]; w_scales [E, N, K/16]; tensor_scales f32 [E].
    w_layout WLAYOUT_KTILE64 when the weight arrays come from moe_pack_weights.
    Returns (Y [R, N] or [R, N/2] for EPI_SILU_GATE, algorithm that ran)."""
    x_rows, K = X.shape
    E, N = w_main.shape[0], w_main.shape[1]
    sparse = w_meta is not None
    _need(X, torch.bfloat16, "X"); _need(expert_offsets, torch.int32, "expert_offsets", (E + 1,))
    if row_token is not None:
        _need(row_token, torch.int32, "row_token", (R,))
    _need(w_main, torch.uint8, "w_main", (E, N, K // 4 if sparse else K // 2))
    if sparse:
        _need(w_meta, torch.uint8, "w_meta", (E, N, K // 8))
    _need(w_scales, torch.uint8, "w_scales", (E, N, K // 16)); _need(tensor_scales, torch.float32, "tensor_scales", (E,))
    ncols = N // 2 if epilogue == EPI_SILU_GATE else N
    Y = Y if Y is not None else torch.empty((R, ncols), dtype=y_dtype, device=X.device)
    dt = SSN_F32 if Y.dtype == torch.float32 else SSN_BF16 if Y.dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError("Y must be float32 or bfloat16")
    _need(Y, Y.dtype, "Y", (R, ncols))
    used = ctypes.c_int(-1)
    cargs = (_ptr(X), x_rows, _ptr(row_token), _ptr(expert_offsets), E, R, N, K, int(sparse), int(w_layout),
             _ptr(w_main), _ptr(w_meta), _ptr(w_scales), _ptr(tensor_scales), epilogue, _ptr(Y), dt, algo,
             ctypes.byref(used), _stream(X.device))
    if prepare:
        return Prepared("moe_grouped_gemm_nvfp4", cargs, (X, row_token, expert_offsets, w_main, w_meta, w_scales,
                                                          tensor_scales, used, Y)), (Y, used)
    _check(lib().moe_grouped_gemm_nvfp4(*cargs))
    return Y, used.value


def moe_pack_ktiles(src, piece_bytes, out=None, prepare=False):
    """64-k tiled copy of one expert weight array [E, N, row_bytes] (uint8): out[e][kt][n] =
    src[e][n][kt*P:(kt+1)*P] with P = piece_bytes (codes 32, vals 16, meta 8, scales 4). The
    result keeps the shape [E, N, row_bytes]; only the byte order inside each expert changes."""
    _need(src, torch.uint8, "src")
    if src.dim() != 3:
        raise ValueError("src must be [E, N, row_bytes]")
    E, N, rb = src.shape
    out = out if out is not None else torch.empty_like(src)
    _need(out, torch.uint8, "out", (E, N, rb))
    cargs = (_ptr(src), E, N, rb, int(piece_bytes), _ptr(out), _stream(src.device))
    return _run("moe_pack_ktiles", cargs, prepare, (src,), out)


def moe_pack_weights(w):
    """(main, meta or None, scales, ts) in the row layout -> the same tuple in the 64-k tiled
    layout (WLAYOUT_KTILE64)."""
    main, meta, scales, ts = w
    sparse = meta is not None
    return (moe_pack_ktiles(main, 16 if sparse else 32), moe_pack_ktiles(meta, 8) if sparse else None,
            moe_pack_ktiles(scales, 4), ts)


def moe_combine(Yd, row_of, topk_weights, out=None, prepare=False):
    """out[t] = sum_j topk_weights[t, j] * Yd[row_of[t*k + j]] (f32 [T, D])."""
    R, D = Yd.shape
    T, k = topk_weights.shape
    dt = SSN_F32 if Yd.dtype == torch.float32 else SSN_BF16 if Yd.dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError("Yd must be float32 or bfloat16")
    _need(Yd, Yd.dtype, "Yd"); _need(row_of, torch.int32, "row_of", (T * k,))
    _need(topk_weights, torch.float32, "topk_weights")
    out = out if out is not None else torch.empty((T, D), dtype=torch.float32, device=Yd.device)
    _need(out, torch.float32, "out", (T, D))
    cargs = (_ptr(Yd), dt, R, _ptr(row_of), _ptr(topk_weights), T, k, D, _ptr(out), _stream(Yd.device))
    return _run("moe_combine", cargs, prepare, (Yd, row_of, topk_weights), out)


def moe_nvfp4_ffn(X, topk_ids, topk_weights, E, up, down, out=None, prepare=False, w_layout=WLAYOUT_ROWS):
    """The whole grouped-expert FFN. up = (main [E, 2I, D/2 or D/4], meta or None, scales
    [E, 2I, D/16], ts [E]); down = (main [E, D, I/2 or I/4], meta or None, scales [E, D, I/16],
    ts [E]); w_layout WLAYOUT_KTILE64 when both come from moe_pack_weights.
    Returns (out f32 [T, D], bad_ids int64 [1] device)."""
    T, D = X.shape
    _, k = topk_ids.shape
    I = up[2].shape[1] // 2
    sparse = up[1] is not None
    _need(X, torch.bfloat16, "X"); _need(topk_ids, torch.int32, "topk_ids", (T, k))
    _need(topk_weights, torch.float32, "topk_weights", (T, k))
    dev = X.device
    out = out if out is not None else torch.empty((T, D), dtype=torch.float32, device=dev)
    bad = torch.empty(1, dtype=torch.int64, device=dev)
    nws = lib().moe_ffn_workspace_bytes(T, k, E, I, D)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    cargs = (_ptr(X), T, D, _ptr(topk_ids), _ptr(topk_weights), k, E, I, int(sparse), int(w_layout), _ptr(up[0]),
             _ptr(up[1]),
             _ptr(up[2]), _ptr(up[3]), _ptr(down[0]), _ptr(down[1]), _ptr(down[2]), _ptr(down[3]), _ptr(out),
             _ptr(bad), _ptr(ws), nws, _stream(dev))
    return _run("moe_nvfp4_ffn", cargs, prepare, (X, topk_ids, topk_weights, up, down, ws), (out, bad))



# ------------------------------------------------------------------------------------------------
# W4A4 variant (MXFP4 activations and weights)


def mxfp4_tiled_bytes(R, K):
    """(code bytes, scale bytes) of the MX_TILED layout of [R, K]."""
    sb = ctypes.c_int64(0)
    cb = lib().mxfp4_tiled_bytes(R, K, ctypes.byref(sb))
    if cb < 0:
        raise ValueError(f"invalid MXFP4 sizes R={R}, K={K}")
    return cb, sb.value


def mxfp4_quantize(V, layout=MX_TILED, codes=None, scales=None, prepare=False):
    """MXFP4 quantisation of V [R, K] (f32 or bf16). Returns (codes, scales) as uint8 tensors:
    [R, K/2] and [R, K/32] for MX_ROWS, flat arrays of mxfp4_tiled_bytes for MX_TILED."""
    R, K = V.shape
    _need(V, V.dtype, "V")
    dev = V.device
    if layout == MX_ROWS:
        cshape, sshape = (R, K // 2), (R, K // 32)
    else:
        cb, sb = mxfp4_tiled_bytes(R, K)
        cshape, sshape = (cb,), (sb,)
    codes = codes if codes is not None else torch.empty(cshape, dtype=torch.uint8, device=dev)
    scales = scales if scales is not None else torch.empty(sshape, dtype=torch.uint8, device=dev)
    _need(codes, torch.uint8, "codes", cshape); _need(scales, torch.uint8, "scales", sshape)
    cargs = (_ptr(V), _wdt(V), R, K, int(layout), _ptr(codes), _ptr(scales), _stream(dev))
    return _run("mxfp4_quantize", cargs, prepare, (V,), (codes, scales))


def gemm_mxfp4(x_codes, x_scales, M, w_codes, w_scales, N, K, y_dtype=torch.float32, algo=ALGO_AUTO, Y=None,
               prepare=False):
    """W4A4 product Y [M, N] = X_hat . W_hat^T from MX_TILED operands. Returns (Y, algorithm)."""
    for t, n, (R, ) in ((x_codes, "x_codes", (M,)), (w_codes, "w_codes", (N,))):
        _need(t, torch.uint8, n, (mxfp4_tiled_bytes(R, K)[0],))
    _need(x_scales, torch.uint8, "x_scales", (mxfp4_tiled_bytes(M, K)[1],))
    _need(w_scales, torch.uint8, "w_scales", (mxfp4_tiled_bytes(N, K)[1],))
    dev = x_codes.device
    Y = Y if Y is not None else torch.empty((M, N), dtype=y_dtype, device=dev)
    dt = SSN_F32 if Y.dtype == torch.float32 else SSN_BF16 if Y.dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError("Y must be float32 or bfloat16")
    _need(Y, Y.dtype, "Y", (M, N))
    used = ctypes.c_int(-1)
    cargs = (_ptr(x_codes), _ptr(x_scales), M, _ptr(w_codes), _ptr(w_scales), N, K, _ptr(Y), dt, algo,
             ctypes.byref(used), _stream(dev))
    if prepare:
        return Prepared("gemm_mxfp4", cargs, (x_codes, x_scales, w_codes, w_scales, used, Y)), (Y, used)
    _check(lib().gemm_mxfp4(*cargs))
    return Y, used.value

def moe_nvfp4_ffn_noalloc(X, topk_ids, topk_weights, E, up, down, out, bad_ids, w_layout=WLAYOUT_ROWS):
    """moe_nvfp4_ffn with the library's static per-GPU workspace instead of a caller-provided
    one: the call itself allocates nothing (out f32 [T, D] and bad_ids int64 [1] are the
    caller's). Routings needing more than the static workspace are refused."""
    T, D = X.shape
    _, k = topk_ids.shape
    I = up[2].shape[1] // 2
    sparse = up[1] is not None
    _need(X, torch.bfloat16, "X"); _need(topk_ids, torch.int32, "topk_ids", (T, k))
    _need(topk_weights, torch.float32, "topk_weights", (T, k))
    _need(out, torch.float32, "out", (T, D)); _need(bad_ids, torch.int64, "bad_ids", (1,))
    _check(lib().moe_nvfp4_ffn_noalloc(_ptr(X), T, D, _ptr(topk_ids), _ptr(topk_weights), k, E, I, int(sparse),
                                       int(w_layout), _ptr(up[0]), _ptr(up[1]), _ptr(up[2]), _ptr(up[3]),
                                       _ptr(down[0]), _ptr(down[1]), _ptr(down[2]), _ptr(down[3]), _ptr(out),
                                       _ptr(bad_ids), _stream(X.device)))
    return out, bad_ids


# ------------------------------------------------------------------------------------------------
# integer 4-bit weights with group scales

_DTYPES = {torch.float32: SSN_F32, torch.bfloat16: SSN_BF16, torch.float16: SSN_F16, torch.uint8: None}
_HALVES = (torch.bfloat16, torch.float16)
_ANY = (torch.float32, torch.bfloat16, torch.float16)
_BYTES = (torch.uint8,)


def _first(t, n, name, allowed):
    """(shape, device, dtype code) of a call's leading tensor, which settles its device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")
    dt = _code(t.dtype, name, allowed)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.shape, t.device, dt


def _size(t, n, name):
    """Shape of a tensor of n dimensions that _on checks later."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} dimensions, got {len(shape)}")
    return shape


def _code(dtype, name, allowed):
    if dtype not in allowed:
        raise TypeError(f"{name} must be one of {', '.join(str(a)[6:] for a in allowed)}, got {dtype}")
    return _DTYPES[dtype]


def _on(dev, t, dtype, name, shape):
    """Address of a contiguous tensor of this type and shape on `dev`."""
    if isinstance(t, torch.Tensor) and t.device == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be a device tensor on {dev}, it is on {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name} must be contiguous")


def _run_on(dev, fname, cargs, prepare, keep, result):
    """_run with `dev` current for the launch and its current stream as the last argument. A prepared call
    launches on the device that is current when it is called."""
    if dev.type != "cuda":
        raise ValueError(f"{fname} takes device tensors, got tensors on {dev}")
    # A small call's time is the host's: the raw handle and device number take 0.1 us, where
    # torch.cuda.current_stream() and current_device() take 2.2.
    cargs = (*cargs, torch._C._cuda_getCurrentRawStream(dev.index))
    if prepare:
        return _run(fname, cargs, True, keep, result)
    call = getattr(_lib or lib(), fname)
    if dev.index == torch._C._cuda_getDevice():
        status = call(*cargs)
    else:
        with torch.cuda.device(dev):
            status = call(*cargs)
    if status:
        _check(status)
    return result


def _int4_group(K, group):
    if isinstance(group, bool) or not isinstance(group, int) or group < 32 or group % 32:
        raise ValueError(f"group must be a positive multiple of 32, got {group}")
    if group >= 1 << 62:                       # the call takes 64 bits
        raise ValueError(f"group={group} is too large (K gives one group per row)")
    return -(-K // group)


def int4_quantize(W, group=128, symmetric=False, scale_dtype=torch.bfloat16, codes=None, scales=None, zeros=None,
                  prepare=False):
    """4-bit codes of W [N, K] (f32, bf16 or f16) with a scale, and unless symmetric a zero point, per `group`
    consecutive k. Returns (codes u8 [N, K/2], scales of scale_dtype [N, ceil(K/group)], zeros u8 of that shape
    or None)."""
    (N, K), dev, wdt = _first(W, 2, "W", _ANY)
    groups = _int4_group(K, group)
    if symmetric and zeros is not None:
        raise ValueError("symmetric quantisation has no zeros")
    codes = codes if codes is not None else W.new_empty((N, K // 2), dtype=torch.uint8)
    scales = scales if scales is not None else W.new_empty((N, groups), dtype=scale_dtype)
    if not symmetric and zeros is None:
        zeros = W.new_empty((N, groups), dtype=torch.uint8)
    sdt = _code(scales.dtype, "scales", _HALVES)
    cargs = (W.data_ptr(), wdt, N, K, group, sdt, _on(dev, codes, torch.uint8, "codes", (N, K // 2)),
             _on(dev, scales, scales.dtype, "scales", (N, groups)),
             None if zeros is None else _on(dev, zeros, torch.uint8, "zeros", (N, groups)))
    return _run_on(dev, "int4_quantize", cargs, prepare, (W,), (codes, scales, zeros))


def int4_dequantize(codes, scales, zeros=None, group=128, out_dtype=torch.float32, out=None, prepare=False):
    """W_hat [N, K] = scales * (codes - zeros) (zeros None: 8), f32, bf16 or f16."""
    (N, Kh), dev, _ = _first(codes, 2, "codes", _BYTES)
    K = 2 * Kh
    groups = _int4_group(K, group)
    sdt = _code(getattr(scales, "dtype", None), "scales", _HALVES)
    out = out if out is not None else codes.new_empty((N, K), dtype=out_dtype)
    odt = _code(out.dtype, "out", _ANY)
    cargs = (codes.data_ptr(), _on(dev, scales, scales.dtype, "scales", (N, groups)), sdt,
             None if zeros is None else _on(dev, zeros, torch.uint8, "zeros", (N, groups)), N, K, group,
             _on(dev, out, out.dtype, "out", (N, K)), odt)
    return _run_on(dev, "int4_dequantize", cargs, prepare, (codes, scales, zeros), out)


def gemv_int4(X, codes, scales, zeros=None, group=128, y_dtype=torch.float32, algo=ALGO_AUTO, Y=None, prepare=False):
    """Y = X . W_hat^T for a few rows of X (bf16 or f16 [M, K]) and integer 4-bit weights: codes u8 [N, K/2],
    scales bf16 or f16 and zeros u8 (or None: 8) [N, ceil(K/group)]. Returns (Y, algorithm that ran)."""
    (M, K), dev, xdt = _first(X, 2, "X", _HALVES)
    groups = _int4_group(K, group)
    N, _ = _size(codes, 2, "codes")
    sdt = _code(getattr(scales, "dtype", None), "scales", _HALVES)
    Y = Y if Y is not None else X.new_empty((M, N), dtype=y_dtype)
    ydt = _code(Y.dtype, "Y", _ANY)
    used = ctypes.c_int(-1)
    cargs = (X.data_ptr(), xdt, M, N, K, _on(dev, codes, torch.uint8, "codes", (N, K // 2)),
             _on(dev, scales, scales.dtype, "scales", (N, groups)), sdt,
             None if zeros is None else _on(dev, zeros, torch.uint8, "zeros", (N, groups)), group,
             _on(dev, Y, Y.dtype, "Y", (M, N)), ydt, algo, ctypes.byref(used))
    out = _run_on(dev, "gemv_int4", cargs, prepare, (X, codes, scales, zeros, used), Y)
    return (out[0], (Y, used)) if prepare else (Y, used.value)


def moe_grouped_gemv_int4(X, row_token, expert_offsets, R, codes, scales, zeros=None, group=128, epilogue=EPI_NONE,
                          y_dtype=torch.float32, algo=ALGO_AUTO, Y=None, prepare=False):
    """Every expert's integer 4-bit product in one launch, for routings with few rows per expert. X bf16 or f16
    [x_rows, K]; row_token int32 [R] or None (identity); expert_offsets int32 [E+1]; codes u8 [E, N, K/2], scales
    bf16 or f16 and zeros u8 (or None: 8) [E, N, ceil(K/group)]. Returns (Y [R, N], or [R, N/2] for
    EPI_SILU_GATE, algorithm that ran); rows of no expert keep what Y held."""
    (x_rows, K), dev, xdt = _first(X, 2, "X", _HALVES)
    groups = _int4_group(K, group)
    E, N, _ = _size(codes, 3, "codes")
    sdt = _code(getattr(scales, "dtype", None), "scales", _HALVES)
    ncols = N // 2 if epilogue == EPI_SILU_GATE else N
    Y = Y if Y is not None else X.new_empty((R, ncols), dtype=y_dtype)
    ydt = _code(Y.dtype, "Y", _ANY)
    used = ctypes.c_int(-1)
    cargs = (X.data_ptr(), xdt, x_rows, None if row_token is None else _on(dev, row_token, torch.int32, "row_token", (R,)),
             _on(dev, expert_offsets, torch.int32, "expert_offsets", (E + 1,)), E, R, N, K,
             _on(dev, codes, torch.uint8, "codes", (E, N, K // 2)),
             _on(dev, scales, scales.dtype, "scales", (E, N, groups)), sdt,
             None if zeros is None else _on(dev, zeros, torch.uint8, "zeros", (E, N, groups)), group, epilogue,
             _on(dev, Y, Y.dtype, "Y", (R, ncols)), ydt, algo, ctypes.byref(used))
    out = _run_on(dev, "moe_grouped_gemv_int4", cargs, prepare,
                  (X, row_token, expert_offsets, codes, scales, zeros, used), Y)
    return (out[0], (Y, used)) if prepare else (Y, used.value)


# ------------------------------------------------------------------------------------------------
# tokens to expert order and back, and the gradients


def _entries(dev, row_of, T, topk_weights):
    """(k, address of row_of [T*k], address of the weights [T, k] or None) of a routing of T tokens."""
    if not isinstance(row_of, torch.Tensor) or row_of.dim() != 1:
        raise ValueError("row_of must be a tensor of one dimension")
    F = row_of.shape[0]
    if topk_weights is not None:
        if not isinstance(topk_weights, torch.Tensor) or topk_weights.dim() != 2:
            raise ValueError("topk_weights must be a tensor of two dimensions")
        k = topk_weights.shape[1]
        w = _on(dev, topk_weights, torch.float32, "topk_weights", (T, k))
    else:
        k, w = F // T if T > 0 else 1, None
    return k, _on(dev, row_of, torch.int32, "row_of", (T * k,)), w


def moe_permute(X, row_of, topk_weights=None, R=None, Xp=None, prepare=False):
    """Tokens to expert order: Xp[row_of[t*k+j]] = topk_weights[t, j] * X[t] (no weights: a copy). X f32, bf16 or
    f16 [T, D]; row_of int32 [T*k] as moe_route gives it (entries outside [0, R) have no row). Returns Xp [R, D]
    of X's type, R = T*k unless given; rows that no entry owns keep what Xp held. Its gradient is
    moe_permute_backward, which nothing calls by itself."""
    (T, D), dev, dt = _first(X, 2, "X", _ANY)
    k, ro, w = _entries(dev, row_of, T, topk_weights)
    R = R if R is not None else (T * k if Xp is None else Xp.shape[0])
    Xp = Xp if Xp is not None else X.new_empty((R, D))
    cargs = (X.data_ptr(), dt, T, k, D, ro, w, R, _on(dev, Xp, X.dtype, "Xp", (R, D)))
    return _run_on(dev, "moe_permute", cargs, prepare, (X, row_of, topk_weights), Xp)


def _dweights(dev, dweights, other, name, dtype, shape, T, k):
    """(address of `other` or None, the weights' gradient or None, its address or None)."""
    if other is None:
        if dweights is not None:
            raise ValueError(f"dweights needs {name}")
        return None, None, None
    dweights = dweights if dweights is not None else torch.empty((T, k), dtype=torch.float32, device=dev)
    return _on(dev, other, dtype, name, shape), dweights, _on(dev, dweights, torch.float32, "dweights", (T, k))


def moe_permute_backward(dXp, row_of, T, topk_weights=None, X=None, dX=None, dweights=None, prepare=False):
    """Gradient of moe_permute for T tokens from dXp [R, D]: (dX [T, D] of dXp's type, dweights f32 [T, k]).
    The weights' gradient needs the forward's X; without X it is None."""
    (R, D), dev, dt = _first(dXp, 2, "dXp", _ANY)
    k, ro, w = _entries(dev, row_of, T, topk_weights)
    dX = dX if dX is not None else dXp.new_empty((T, D))
    x, dweights, dw = _dweights(dev, dweights, X, "X", dXp.dtype, (T, D), T, k)
    cargs = (dXp.data_ptr(), dt, R, ro, w, T, k, D, x, _on(dev, dX, dXp.dtype, "dX", (T, D)), dw)
    return _run_on(dev, "moe_permute_backward", cargs, prepare, (dXp, row_of, topk_weights, X), (dX, dweights))


def moe_unpermute(Yp, row_of, T, topk_weights=None, out_dtype=None, out=None, prepare=False):
    """Expert rows back to T tokens: out[t] = sum_j topk_weights[t, j] * Yp[row_of[t*k+j]] (no weights: the plain
    sum), summed in f32. Yp f32, bf16 or f16 [R, D]; out [T, D] of Yp's type unless out_dtype is float32. Its
    gradient is moe_unpermute_backward, which nothing calls by itself."""
    (R, D), dev, ydt = _first(Yp, 2, "Yp", _ANY)
    k, ro, w = _entries(dev, row_of, T, topk_weights)
    if out is None:
        out = Yp.new_empty((T, D), dtype=out_dtype)
    odt = _code(out.dtype, "out", (torch.float32, Yp.dtype))
    cargs = (Yp.data_ptr(), ydt, R, ro, w, T, k, D, _on(dev, out, out.dtype, "out", (T, D)), odt)
    return _run_on(dev, "moe_unpermute", cargs, prepare, (Yp, row_of, topk_weights), out)


def moe_unpermute_backward(dout, row_of, R, topk_weights=None, Yp=None, y_dtype=None, dYp=None, dweights=None,
                           prepare=False):
    """Gradient of moe_unpermute (and of moe_combine) from dout [T, D]: (dYp [R, D], dweights f32 [T, k]). dYp has
    y_dtype (dout's type unless given), or Yp's type; the weights' gradient needs the forward's Yp; without Yp it
    is None. Rows that no entry owns keep what dYp held."""
    (T, D), dev, odt = _first(dout, 2, "dout", _ANY)
    k, ro, w = _entries(dev, row_of, T, topk_weights)
    if y_dtype is None:
        y_dtype = Yp.dtype if Yp is not None else dYp.dtype if dYp is not None else dout.dtype
    ydt = _code(y_dtype, "dYp", _ANY)
    _code(dout.dtype, "dout", (torch.float32, y_dtype))
    dYp = dYp if dYp is not None else dout.new_empty((R, D), dtype=y_dtype)
    y, dweights, dw = _dweights(dev, dweights, Yp, "Yp", y_dtype, (R, D), T, k)
    cargs = (dout.data_ptr(), odt, T, k, D, ro, w, R, y, _on(dev, dYp, y_dtype, "dYp", (R, D)), ydt, dw)
    return _run_on(dev, "moe_unpermute_backward", cargs, prepare, (dout, row_of, topk_weights, Yp), (dYp, dweights))


# ------------------------------------------------------------------------------------------------
# 4-bit cache of keys and values, and attention over it


class KvNvfp4(NamedTuple):
    """A cache of keys and values in NVFP4: pages of page_size tokens (a multiple of 16), heads of width D (a multiple of
    32, at most 256). The tensors are the caller's; kv_nvfp4_empty makes them."""
    k_codes: torch.Tensor           # u8 [pages, Hkv, page_size, D/2]
    k_scales: torch.Tensor          # u8 [pages, Hkv, page_size, D/16]
    v_codes: torch.Tensor           # u8 [pages, Hkv, page_size, D/2]
    v_scales: torch.Tensor          # u8 [pages, Hkv, D/16, page_size]
    k_tensor_scale: torch.Tensor    # f32 [Hkv]
    v_tensor_scale: torch.Tensor    # f32 [Hkv]


def kv_nvfp4_empty(pages, page_size, D, k_tensor_scale, v_tensor_scale):
    """An unwritten cache for the heads' tensor scales (f32 [Hkv] device tensors: the largest magnitude of a head over
    2688, from calibration or from its first tokens)."""
    H, new = k_tensor_scale.shape[0], k_tensor_scale.new_empty
    u8 = dict(dtype=torch.uint8)
    return KvNvfp4(new((pages, H, page_size, D // 2), **u8), new((pages, H, page_size, D // 16), **u8),
                   new((pages, H, page_size, D // 2), **u8), new((pages, H, D // 16, page_size), **u8),
                   k_tensor_scale, v_tensor_scale)


def _kv(dev, cache):
    """(addresses of the cache's tensors, (pages, page_size, Hkv, D)). One combined check, 1.8 us; six by _on take 2.1
    of a call's 8."""
    kc, ks, vc, vs, kt, vt = cache
    P, H, S, Dh = _size(kc, 4, "k_codes")
    D, u8, f32 = 2 * Dh, torch.uint8, torch.float32
    try:
        at = dev.index if dev.type == "cuda" else -1
        if (kc.dtype is u8 and ks.dtype is u8 and vc.dtype is u8 and vs.dtype is u8 and kt.dtype is f32 and vt.dtype is f32
                and kc.get_device() == at and ks.get_device() == at and vc.get_device() == at and vs.get_device() == at
                and kt.get_device() == at and vt.get_device() == at
                and vc.shape == kc.shape and ks.shape == (P, H, S, D // 16) and vs.shape == (P, H, D // 16, S)
                and kt.shape == (H,) and vt.shape == (H,)
                and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()
                and kt.is_contiguous() and vt.is_contiguous()):
            return (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), kt.data_ptr(), vt.data_ptr()), (P, S, H, D)
    except AttributeError:
        pass                                       # something that is no tensor: named below
    return (_on(dev, kc, u8, "k_codes", (P, H, S, Dh)), _on(dev, ks, u8, "k_scales", (P, H, S, D // 16)),
            _on(dev, vc, u8, "v_codes", (P, H, S, Dh)), _on(dev, vs, u8, "v_scales", (P, H, D // 16, S)),
            _on(dev, kt, f32, "k_tensor_scale", (H,)), _on(dev, vt, f32, "v_tensor_scale", (H,))), (P, S, H, D)


def _rows(dev, t, dtype, name, shape):
    """(address, stride of a token, stride of a head) of a tensor whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be a device tensor on {dev}, it is on {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    token, head, one = t.stride()
    if shape[0] == 0:                              # no rows: whatever strides it has
        return t.data_ptr(), 0, 0
    if one != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), token if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def kv_nvfp4_append(K, V, slots, cache, bad_slots=None, prepare=False):
    """Quantise keys and values [T, Hkv, D] (f32, bf16 or f16, one type; rows may be strided) into the cache: token t goes
    to slots[t] (int64 [T] device: page * page_size + place; negative: nowhere). bad_slots (int64 [1] device), where
    given, receives the count of slots beyond the cache. Returns the cache."""
    T = _size(K, 3, "K")[0]
    dev = K.device
    at, (P, S, H, D) = _kv(dev, cache)
    k, kt, kh = _rows(dev, K, K.dtype, "K", (T, H, D))
    v, vt, vh = _rows(dev, V, K.dtype, "V", (T, H, D))
    cargs = (k, v, _code(K.dtype, "K", _ANY), T, kt, kh, vt, vh, _on(dev, slots, torch.int64, "slots", (T,)), *at, P, S, H,
             D, None if bad_slots is None else _on(dev, bad_slots, torch.int64, "bad_slots", (1,)))
    return _run_on(dev, "kv_nvfp4_append", cargs, prepare, (K, V, slots, bad_slots), cache)


def kv_nvfp4_read(slots, cache, out_dtype=torch.bfloat16, K=None, V=None, prepare=False):
    """The cached keys and values of any slots (int64 [T] device): (K, V) [T, Hkv, D] of out_dtype (f32, bf16 or f16);
    zeros where a slot is negative or beyond the cache."""
    (T,) = _size(slots, 1, "slots")
    dev = slots.device
    at, (P, S, H, D) = _kv(dev, cache)
    if K is None:
        K = slots.new_empty((T, H, D), dtype=out_dtype)
        k = K.data_ptr()
    else:
        k = _on(dev, K, K.dtype, "K", (T, H, D))
    dt = _code(K.dtype, "K", _ANY)
    if V is None:
        V = torch.empty_like(K)
        v = V.data_ptr()
    else:
        v = _on(dev, V, K.dtype, "V", (T, H, D))
    cargs = (_on(dev, slots, torch.int64, "slots", (T,)), T, *at, P, S, H, D, k, v, dt)
    return _run_on(dev, "kv_nvfp4_read", cargs, prepare, (slots, cache), (K, V))


def attn_kv_nvfp4(Q, cache, block_table, seq_lens, q_offsets=None, max_q=None, max_kv=None, scale=None, causal=True,
                  window=0, out_dtype=None, with_lse=False, algo=ALGO_AUTO, out=None, lse=None, workspace=None,
                  prepare=False):
    """Attention of B sequences' newest tokens over the cache, their own keys and values in it already. Q bf16 or f16
    [Tq, Hq, D] (rows may be strided), Hq a multiple of the cache's heads; block_table int32 [B, blocks]; seq_lens int32
    [B], the queries' tokens included; q_offsets int32 [B+1] where sequences have different numbers of queries (else
    Tq / B each). max_q and max_kv bound a sequence's queries and tokens (host numbers that size the launch: Tq, or
    Tq / B, and the table's width unless given). max_q chooses the kernel of the whole batch too: with q_offsets give it (32
    single tokens over 8192 keys take 57 us with max_q=1, 149 without), and give a prompt's chunk and decoded tokens
    calls of their own. scale: 1 / sqrt(D) unless given. window > 0: a query keeps its last
    `window` keys. Returns (out [Tq, Hq, D] of Q's type unless out_dtype is float32, lse f32 [Tq, Hq] if with_lse or
    given else None, algorithm that ran); rows of no sequence keep what out held, rows without keys are 0,
    rows of queries that are not finite NaN."""
    (Tq, Hq, D) = _size(Q, 3, "Q")
    dev, qdt = Q.device, _code(Q.dtype, "Q", _HALVES)
    at, (P, S, H, Dc) = _kv(dev, cache)
    q, qt, qh = _rows(dev, Q, Q.dtype, "Q", (Tq, Hq, Dc))
    B, blocks = _size(block_table, 2, "block_table")
    if max_q is None:
        max_q = Tq if q_offsets is not None else Tq // B if B else 0
    if max_kv is None:
        max_kv = min(blocks * S, 1 << 27)
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = Q.new_empty((Tq, Hq, D), dtype=out_dtype)
        o = out.data_ptr()
    else:
        o = _on(dev, out, out.dtype, "out", (Tq, Hq, D))
    odt = _code(out.dtype, "out", (torch.float32, Q.dtype))
    if lse is None and with_lse:
        lse = Q.new_empty((Tq, Hq), dtype=torch.float32)
    L = _lib or lib()
    if dev.type == "cuda" and dev.index != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            nws = L.attn_kv_nvfp4_workspace_bytes(B, Hq, H, D, max_q, max_kv)
    else:
        nws = L.attn_kv_nvfp4_workspace_bytes(B, Hq, H, D, max_q, max_kv)
    if nws < 0:
        _check(SSN_E_SHAPE)
    if workspace is not None:
        ws, nws = _on(dev, workspace, torch.uint8, "workspace", workspace.shape), workspace.numel()
    elif nws:
        workspace = Q.new_empty(nws, dtype=torch.uint8)
        ws = workspace.data_ptr()
    else:
        ws = None
    used = ctypes.c_int(-1)
    cargs = (q, qdt, Tq, Hq, qt, qh, *at, P, S, H, D, _on(dev, block_table, torch.int32, "block_table", (B, blocks)), B,
             blocks, _on(dev, seq_lens, torch.int32, "seq_lens", (B,)),
             None if q_offsets is None else _on(dev, q_offsets, torch.int32, "q_offsets", (B + 1,)), max_q, max_kv, scale,
             causal, window, o, odt, None if lse is None else _on(dev, lse, torch.float32, "lse", (Tq, Hq)), algo,
             ctypes.byref(used), ws, nws)
    res = _run_on(dev, "attn_kv_nvfp4", cargs, prepare,
                  (Q, cache, block_table, seq_lens, q_offsets, workspace, used), (out, lse))
    return (res[0], (out, lse, used)) if prepare else (out, lse, used.value)


def mfma_probe_sink_floats():
    return int(lib().mfma_probe_sink_floats())


def mfma_probe(kind, waves_per_simd, iters, sink, seed=0, stream_device=None):
    """Calibration launch (see include/ssnvfp4.h): register-resident matrix ops on random
    operands. Returns the launch's floating-point operations; the caller times it."""
    fl = ctypes.c_double(0.0)
    _need(sink, torch.float32, "sink")
    if sink.numel() < mfma_probe_sink_floats():
        raise ValueError(f"sink needs {mfma_probe_sink_floats()} floats")
    _check(lib().mfma_probe(kind, waves_per_simd, iters, seed & 0xFFFFFFFF, _ptr(sink), ctypes.byref(fl),
                            _stream(sink.device)))
    return fl.value
