"""Thin ctypes binding over libcsa.so.

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels.  torch supplies device memory and the current stream.  The
functions carry the C names of include/csa.h and return the status code after
raising ``CSAError`` on a failure; outputs are written into the caller's
tensors.  Importing this module loads the library and fails loudly if it has
not been built (``compressed_sparse_attention_compress_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "csa.h")

CSA_BF16, CSA_FP32 = 0, 1
STATUS = {0: "CSA_OK", -1: "CSA_ERR_INVALID_ARG", -2: "CSA_ERR_UNSUPPORTED", -3: "CSA_ERR_WORKSPACE",
          -4: "CSA_ERR_CUDA", -5: "CSA_ERR_DEVICE_TIMEOUT", -6: "CSA_ERR_DEVICE_BOUNDS"}


class CSAError(RuntimeError):
    def __init__(self, name, code):
        super().__init__(f"{name} failed: {STATUS.get(code, code)}")
        self.code = code


def declared_symbols(header: str = HEADER) -> list:
    """Names of the functions include/csa.h declares."""
    text = open(header).read()
    return re.findall(r"^(?:csa_status_t|size_t|const char\*)\s+(\w+)\s*\(", text, flags=re.M)


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m compressed_sparse_attention_compress_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    sig = {
        "csa_create": [I, P],
        "csa_destroy": [P],
        "csa_get_device_status": [P, P, P],
        "csa_set_position_offsets": [P, P, I],
        "csa_compressed_offsets": [P, P, I, I, P, P],
        "csa_compress": [P, P, P, P, P, P, I, I, I, I, I, I, I, P, P],
        "csa_compress_pair": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P],
        "csa_compress_ex": [P, P, P, P, P, P, P, F, I, F, I, I, P, P, I, I, I, I, I, I, I, P, P],
        "csa_indexer_topk": [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, P],
        "csa_sparse_attn_fwd": [P, P, P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, F, I, P, P, P, P],
        "hca_attn_fwd": [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, P, P, P],
        "window_attn_fwd": [P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P],
        "csa_sparse_attn_bwd": [P, P, P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, F, I, P, P, P, P, P, P, P, P,
                                P, P, P],
        "hca_attn_bwd": [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, P, P, P, P, P, P, P, P, P, P],
        "window_attn_bwd": [P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P, P, P, P, P, P, P],
        "csa_indexer_kl_bwd": [P, P, P, P, P, P, P, I, P, P, P, P, I, I, I, I, I, I, I, I, F, F, I, P, P, P, P],
        "csa_indexer_kl_ex": [P, P, P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, I, F, I, P, P, P, P, Z, P, P, P],
        "csa_quantize_fp8": [P, P, ctypes.c_int64, I, I, P, P, P],
        "csa_indexer_topk_fp8": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, P],
        "csa_indexer_kl": [P, P, P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, I, F, I, P, P, P, P, Z, P],
        "csa_cache_write": [P, P, P, P, P, P, I, I, I, P],
        "csa_cache_read": [P, P, P, P, I, I, I, P, P, P],
        "csa_cache_attn_fwd": [P, P, P, P, P, I, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P, Z, P],
        "csa_indexer_kl_static_scratch": [P, P, P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, I, I, F, I, P, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = I
    lib.csa_status_string.argtypes = [I]
    lib.csa_status_string.restype = ctypes.c_char_p
    lib.csa_indexer_kl_workspace.argtypes = [I]
    lib.csa_indexer_kl_workspace.restype = Z
    lib.csa_cache_attn_workspace.argtypes = [P, I, I, I, I]
    lib.csa_cache_attn_workspace.restype = Z
    return lib


LIB = _load()


def _p(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libcsa must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t) -> int:
    if t.dtype == torch.bfloat16:
        return CSA_BF16
    if t.dtype == torch.float32:
        return CSA_FP32
    raise TypeError(f"unsupported activation dtype {t.dtype}")


def _check(name, code):
    if code != 0:
        raise CSAError(name, code)
    return code


class Handle:
    """Owns a csa_handle_t (device properties + device status word)."""

    def __init__(self, device: int = 0):
        h = ctypes.c_void_p()
        _check("csa_create", LIB.csa_create(int(device), ctypes.byref(h)))
        self._h = h
        self.device = device

    @property
    def ptr(self):
        return self._h

    def device_status(self, stream=None) -> int:
        v = ctypes.c_int(0)
        _check("csa_get_device_status", LIB.csa_get_device_status(self._h, _stream(stream), ctypes.byref(v)))
        return v.value

    def set_position_offsets(self, pos0=None, cmp_rows: int = 0):
        """Per-sequence position of the first packed row (device int32 [B]) for the
        query calls made with this handle from now on; None restores 0."""
        _check("csa_set_position_offsets", LIB.csa_set_position_offsets(self._h, _p(pos0), int(cmp_rows)))

    def close(self):
        if self._h:
            LIB.csa_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def csa_compressed_offsets(h: Handle, cu_seqlens, ratio: int, cu_cmp, stream=None):
    B = cu_seqlens.numel() - 1
    return _check("csa_compressed_offsets",
                  LIB.csa_compressed_offsets(h.ptr, _p(cu_seqlens), B, int(ratio), _p(cu_cmp), _stream(stream)))


def csa_compress(h: Handle, x, z, pos_bias, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int, overlap: bool,
                 out, stream=None):
    T_cap, D = x.shape
    return _check("csa_compress", LIB.csa_compress(
        h.ptr, _p(x), _p(z), _p(pos_bias), _p(cu_seqlens), _p(cu_cmp), cu_seqlens.numel() - 1, T_cap,
        int(max_seqlen), D, int(ratio), int(bool(overlap)), _dtype(x), _p(out), _stream(stream)))


def csa_compress_pair(h: Handle, x_kv, z_kv, pos_bias_kv, x_I, z_I, pos_bias_I, cu_seqlens, max_seqlen: int,
                      ratio: int, overlap: bool, cu_cmp, kv_cmp, kI_cmp, stream=None):
    """Both compressors of a layer and the compressed offsets in one launch."""
    T_cap, D = x_kv.shape
    d_I = x_I.shape[1]
    return _check("csa_compress_pair", LIB.csa_compress_pair(
        h.ptr, _p(x_kv), _p(z_kv), _p(pos_bias_kv), _p(x_I), _p(z_I), _p(pos_bias_I), _p(cu_seqlens),
        cu_seqlens.numel() - 1, T_cap, int(max_seqlen), D, d_I, int(ratio), int(bool(overlap)), _dtype(x_kv),
        _p(cu_cmp), _p(kv_cmp), _p(kI_cmp), _stream(stream)))


def csa_compress_ex(h: Handle, x, z, pos_bias, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int, overlap: bool,
                    out, x_prev=None, z_prev=None, norm_weight=None, norm_eps: float = 1e-6, rope_dim: int = 0,
                    rope_theta: float = 10000.0, rope_pos_stride: int = 1, rope_pos_offset: int = 0, stream=None):
    T_cap, D = x.shape
    return _check("csa_compress_ex", LIB.csa_compress_ex(
        h.ptr, _p(x), _p(z), _p(x_prev), _p(z_prev), _p(pos_bias), _p(norm_weight), float(norm_eps),
        int(rope_dim), float(rope_theta), int(rope_pos_stride), int(rope_pos_offset), _p(cu_seqlens),
        _p(cu_cmp), cu_seqlens.numel() - 1, T_cap, int(max_seqlen), D, int(ratio), int(bool(overlap)),
        _dtype(x), _p(out), _stream(stream)))


def csa_indexer_topk(h: Handle, qI, w, kI, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int, topk: int, idx,
                     stream=None):
    T_cap, H_I, d_I = qI.shape
    k_pad = idx.shape[1]
    return _check("csa_indexer_topk", LIB.csa_indexer_topk(
        h.ptr, _p(qI), _p(w), _p(kI), _p(cu_seqlens), _p(cu_cmp), cu_seqlens.numel() - 1, T_cap,
        int(max_seqlen), H_I, d_I, int(ratio), int(topk), k_pad, _dtype(qI), _p(idx), _stream(stream)))


def csa_sparse_attn_fwd(h: Handle, q, kv_cmp, kv_raw, idx, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int,
                        window: int, softmax_scale: float, out, lse, lse_cmp=None, v_cmp=None, v_raw=None,
                        sink=None, stream=None):
    T_cap, H, d = q.shape
    return _check("csa_sparse_attn_fwd", LIB.csa_sparse_attn_fwd(
        h.ptr, _p(q), _p(kv_cmp), _p(v_cmp), _p(kv_raw), _p(v_raw), _p(idx), idx.shape[1], _p(sink),
        _p(cu_seqlens), _p(cu_cmp), cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, int(ratio),
        int(window), float(softmax_scale), _dtype(q), _p(out), _p(lse), _p(lse_cmp), _stream(stream)))


def hca_attn_fwd(h: Handle, q, kv_cmp, kv_raw, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int, window: int,
                 softmax_scale: float, out, lse, lse_cmp=None, v_cmp=None, v_raw=None, sink=None, stream=None):
    T_cap, H, d = q.shape
    return _check("hca_attn_fwd", LIB.hca_attn_fwd(
        h.ptr, _p(q), _p(kv_cmp), _p(v_cmp), _p(kv_raw), _p(v_raw), _p(sink), _p(cu_seqlens), _p(cu_cmp),
        cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, int(ratio), int(window), float(softmax_scale),
        _dtype(q), _p(out), _p(lse), _p(lse_cmp), _stream(stream)))


def window_attn_fwd(h: Handle, q, kv_raw, cu_seqlens, max_seqlen: int, window: int, softmax_scale: float, out,
                    lse, v_raw=None, sink=None, stream=None):
    T_cap, H, d = q.shape
    return _check("window_attn_fwd", LIB.window_attn_fwd(
        h.ptr, _p(q), _p(kv_raw), _p(v_raw), _p(sink), _p(cu_seqlens), cu_seqlens.numel() - 1, T_cap,
        int(max_seqlen), H, d, int(window), float(softmax_scale), _dtype(q), _p(out), _p(lse), _stream(stream)))


def csa_sparse_attn_bwd(h: Handle, q, kv_cmp, kv_raw, idx, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int,
                        window: int, softmax_scale: float, out, lse, dout, dq, dkv_cmp, dkv_raw, delta,
                        v_cmp=None, v_raw=None, dv_cmp=None, dv_raw=None, sink=None, dsink=None, stream=None):
    T_cap, H, d = q.shape
    return _check("csa_sparse_attn_bwd", LIB.csa_sparse_attn_bwd(
        h.ptr, _p(q), _p(kv_cmp), _p(v_cmp), _p(kv_raw), _p(v_raw), _p(idx), idx.shape[1], _p(sink),
        _p(cu_seqlens), _p(cu_cmp), cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, int(ratio),
        int(window), float(softmax_scale), _dtype(q), _p(out), _p(lse), _p(dout), _p(dq), _p(dkv_cmp),
        _p(dv_cmp), _p(dkv_raw), _p(dv_raw), _p(dsink), _p(delta), _stream(stream)))


def hca_attn_bwd(h: Handle, q, kv_cmp, kv_raw, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int, window: int,
                 softmax_scale: float, out, lse, dout, dq, dkv_cmp, dkv_raw, delta, v_cmp=None, v_raw=None,
                 dv_cmp=None, dv_raw=None, sink=None, dsink=None, stream=None):
    T_cap, H, d = q.shape
    return _check("hca_attn_bwd", LIB.hca_attn_bwd(
        h.ptr, _p(q), _p(kv_cmp), _p(v_cmp), _p(kv_raw), _p(v_raw), _p(sink), _p(cu_seqlens), _p(cu_cmp),
        cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, int(ratio), int(window), float(softmax_scale),
        _dtype(q), _p(out), _p(lse), _p(dout), _p(dq), _p(dkv_cmp), _p(dv_cmp), _p(dkv_raw), _p(dv_raw),
        _p(dsink), _p(delta), _stream(stream)))


def window_attn_bwd(h: Handle, q, kv_raw, cu_seqlens, max_seqlen: int, window: int, softmax_scale: float, out,
                    lse, dout, dq, dkv_raw, delta, v_raw=None, dv_raw=None, sink=None, dsink=None, stream=None):
    T_cap, H, d = q.shape
    return _check("window_attn_bwd", LIB.window_attn_bwd(
        h.ptr, _p(q), _p(kv_raw), _p(v_raw), _p(sink), _p(cu_seqlens), cu_seqlens.numel() - 1, T_cap,
        int(max_seqlen), H, d, int(window), float(softmax_scale), _dtype(q), _p(out), _p(lse), _p(dout), _p(dq),
        _p(dkv_raw), _p(dv_raw), _p(dsink), _p(delta), _stream(stream)))


def csa_indexer_kl_workspace(T_cap: int) -> int:
    return int(LIB.csa_indexer_kl_workspace(int(T_cap)))


def csa_indexer_kl(h: Handle, q, kv_cmp, qI, w, kI, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int,
                   softmax_scale: float, kl_sum, ws, idx=None, lse_cmp=None, kl_per_query=None, n_valid=None,
                   stream=None):
    T_cap, H, d = q.shape
    _, H_I, d_I = qI.shape
    k_pad = idx.shape[1] if idx is not None else 0
    return _check("csa_indexer_kl", LIB.csa_indexer_kl(
        h.ptr, _p(q), _p(kv_cmp), _p(qI), _p(w), _p(kI), _p(idx), k_pad, _p(lse_cmp), _p(cu_seqlens),
        _p(cu_cmp), cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, H_I, d_I, int(ratio),
        float(softmax_scale), _dtype(q), _p(kl_sum), _p(kl_per_query), _p(n_valid), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def csa_indexer_kl_ex(h: Handle, q, kv_cmp, qI, w, kI, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int,
                      softmax_scale: float, kl_sum, ws, teacher_lse=None, student_lse=None, idx=None, lse_cmp=None,
                      kl_per_query=None, n_valid=None, stream=None):
    T_cap, H, d = q.shape
    _, H_I, d_I = qI.shape
    k_pad = idx.shape[1] if idx is not None else 0
    return _check("csa_indexer_kl_ex", LIB.csa_indexer_kl_ex(
        h.ptr, _p(q), _p(kv_cmp), _p(qI), _p(w), _p(kI), _p(idx), k_pad, _p(lse_cmp), _p(cu_seqlens),
        _p(cu_cmp), cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, H_I, d_I, int(ratio),
        float(softmax_scale), _dtype(q), _p(kl_sum), _p(kl_per_query), _p(n_valid), _p(ws),
        ws.numel() * ws.element_size(), _p(teacher_lse), _p(student_lse), _stream(stream)))


def csa_indexer_kl_static_scratch(h: Handle, q, kv_cmp, qI, w, kI, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int,
                                  softmax_scale: float, kl_sum, idx=None, lse_cmp=None, kl_per_query=None,
                                  n_valid=None, stream=None):
    """csa_indexer_kl without a workspace argument: the library's own static
    device scratch is used (for callers that cannot allocate device memory)."""
    T_cap, H, d = q.shape
    _, H_I, d_I = qI.shape
    k_pad = idx.shape[1] if idx is not None else 0
    return _check("csa_indexer_kl_static_scratch", LIB.csa_indexer_kl_static_scratch(
        h.ptr, _p(q), _p(kv_cmp), _p(qI), _p(w), _p(kI), _p(idx), k_pad, _p(lse_cmp), _p(cu_seqlens),
        _p(cu_cmp), cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, H_I, d_I, int(ratio),
        float(softmax_scale), _dtype(q), _p(kl_sum), _p(kl_per_query), _p(n_valid), _stream(stream)))


def csa_indexer_kl_bwd(h: Handle, q, kv_cmp, qI, w, kI, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int,
                       softmax_scale: float, dqI, dw, dkI, idx=None, lse_cmp=None, grad_scale: float = 1.0,
                       student_lse=None, stream=None):
    T_cap, H, d = q.shape
    _, H_I, d_I = qI.shape
    k_pad = idx.shape[1] if idx is not None else 0
    return _check("csa_indexer_kl_bwd", LIB.csa_indexer_kl_bwd(
        h.ptr, _p(q), _p(kv_cmp), _p(qI), _p(w), _p(kI), _p(idx), k_pad, _p(lse_cmp), _p(student_lse),
        _p(cu_seqlens), _p(cu_cmp), cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H, d, H_I, d_I, int(ratio),
        float(softmax_scale), float(grad_scale), _dtype(q), _p(dqI), _p(dw), _p(dkI), _stream(stream)))


def csa_quantize_fp8(h: Handle, x, codes, scales, stream=None):
    """E4M3 codes (uint8, x's shape) and per-row scales (float32, x.shape[:-1]) of x."""
    cols = x.shape[-1]
    return _check("csa_quantize_fp8", LIB.csa_quantize_fp8(
        h.ptr, _p(x), x.numel() // cols, cols, _dtype(x), _p(codes), _p(scales), _stream(stream)))


def csa_indexer_topk_fp8(h: Handle, qI, qI_scale, w, kI, kI_scale, cu_seqlens, cu_cmp, max_seqlen: int, ratio: int,
                         topk: int, idx, stream=None):
    T_cap, H_I, d_I = qI.shape
    return _check("csa_indexer_topk_fp8", LIB.csa_indexer_topk_fp8(
        h.ptr, _p(qI), _p(qI_scale), _p(w), _p(kI), _p(kI_scale), _p(cu_seqlens), _p(cu_cmp),
        cu_seqlens.numel() - 1, T_cap, int(max_seqlen), H_I, d_I, int(ratio), int(topk), idx.shape[1],
        _dtype(w), _p(idx), _stream(stream)))


# ---- serving: the paged 8-bit cache ----------------------------------------
class _CacheStruct(ctypes.Structure):
    """csa_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p), ("n_blocks", ctypes.c_int),
                ("max_blocks", ctypes.c_int), ("block", ctypes.c_int), ("H_kv", ctypes.c_int), ("d", ctypes.c_int)]


def _want(what, t, dtype, shape, device):
    """Address of t: a contiguous tensor of this type and shape on this device (one short test when it is)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{what}: {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{what}: on {t.device}, expected cuda:{device}")
    raise ValueError(f"{what}: tensors passed to libcsa must be contiguous")


class Cache:
    """A paged E4M3 cache over the caller's tensors (held, not copied).

    k (and v, unless V = K): uint8 [n_blocks, H_kv, block, d]; k_scale, v_scale:
    float32 [n_blocks, H_kv]; table: int32 [B, max_blocks], the blocks of each
    sequence in order.  Rows of ``table`` may be rewritten in place between calls.
    """

    def __init__(self, k, k_scale, table, v=None, v_scale=None):
        if not k.is_cuda:
            raise ValueError("k: the cache lives on a CUDA device")
        if (v is None) != (v_scale is None):
            raise ValueError("v and v_scale come together")
        n, H_kv, block, d = k.shape
        dev = k.get_device()
        s = _CacheStruct()
        s.k = _want("k", k, torch.uint8, (n, H_kv, block, d), dev)
        s.k_scale = _want("k_scale", k_scale, torch.float32, (n, H_kv), dev)
        if table.dim() != 2:
            raise ValueError(f"table: shape {tuple(table.shape)}, expected [B, max_blocks]")
        s.table = _want("table", table, torch.int32, table.shape, dev)
        if v is not None:
            s.v = _want("v", v, torch.uint8, (n, H_kv, block, d), dev)
            s.v_scale = _want("v_scale", v_scale, torch.float32, (n, H_kv), dev)
        s.n_blocks, s.max_blocks, s.block, s.H_kv, s.d = n, table.shape[1], block, H_kv, d
        self.k, self.k_scale, self.table, self.v, self.v_scale = k, k_scale, table, v, v_scale
        self.device, self.B, self.H_kv, self.d = dev, table.shape[0], H_kv, d
        self._struct = s
        self._ref = ctypes.addressof(s)


def _stream_of(h, stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(h.device)


def _packing(h, caches, cu_seqlens, pos0):
    """Checked sequences of a cache call: (B, cu pointer, pos0 pointer)."""
    B = cu_seqlens.shape[0] - 1
    for c in caches:
        if c.device != h.device:
            raise ValueError(f"cache on cuda:{c.device}, handle on cuda:{h.device}")
        if not 0 <= B <= c.B:
            raise ValueError(f"table has {c.B} rows for {B} sequences")
    return (B, _want("cu_seqlens", cu_seqlens, torch.int32, (B + 1,), h.device),
            _want("pos0", pos0, torch.int32, (B,), h.device))


def csa_cache_write(h: Handle, cache: Cache, x_k, cu_seqlens, pos0, x_v=None, stream=None):
    """Quantise rows [T_cap, H_kv, d] into the cache at positions pos0[b] + i."""
    B, cu, p0 = _packing(h, (cache,), cu_seqlens, pos0)
    shape = (x_k.shape[0], cache.H_kv, cache.d)
    k = _want("x_k", x_k, x_k.dtype, shape, h.device)
    v = _want("x_v", x_v, x_k.dtype, shape, h.device) if x_v is not None else None
    return _check("csa_cache_write", LIB.csa_cache_write(
        h.ptr, cache._ref, k, v, cu, p0, B, shape[0], _dtype(x_k), _stream_of(h, stream)))


def csa_cache_read(h: Handle, cache: Cache, cu_seqlens, pos0, k_out, v_out=None, stream=None):
    """Rows at positions pos0[b] + i of the cache, dequantised into [T_cap, H_kv, d]."""
    B, cu, p0 = _packing(h, (cache,), cu_seqlens, pos0)
    shape = (k_out.shape[0], cache.H_kv, cache.d)
    k = _want("k_out", k_out, k_out.dtype, shape, h.device)
    v = _want("v_out", v_out, k_out.dtype, shape, h.device) if v_out is not None else None
    return _check("csa_cache_read", LIB.csa_cache_read(
        h.ptr, cache._ref, cu, p0, B, shape[0], _dtype(k_out), k, v, _stream_of(h, stream)))


def csa_cache_attn_workspace(h: Handle, T_cap: int, H: int, H_kv: int, d: int) -> int:
    return int(LIB.csa_cache_attn_workspace(h.ptr, int(T_cap), int(H), int(H_kv), int(d)))


def csa_cache_attn_fwd(h: Handle, q, cu_seqlens, pos0, softmax_scale: float, out, ws, cmp=None, raw=None, idx=None,
                       cu_cmp=None, ratio: int = 0, window: int = 0, sink=None, lse=None, stream=None):
    """Attention of q [T_cap, H, d] over a cache of compressed entries (all visible ones, or
    idx's) and the last ``window`` rows of a raw cache, in one softmax."""
    caches = [c for c in (cmp, raw) if c is not None]
    if not caches:
        raise ValueError("neither cmp nor raw is given")
    B, cu, p0 = _packing(h, caches, cu_seqlens, pos0)
    dev = h.device
    shape = q.shape
    T, H, d = shape
    k_pad, i, cc, sk, ls, w, n = 0, None, None, None, None, None, 0
    if idx is not None:
        k_pad = idx.shape[-1]
        i = _want("idx", idx, torch.int32, (T, k_pad), dev)
    if cu_cmp is not None:
        cc = _want("cu_cmp", cu_cmp, torch.int32, (B + 1,), dev)
    if sink is not None:
        sk = _want("sink", sink, torch.float32, (H,), dev)
    if lse is not None:
        ls = _want("lse", lse, torch.float32, (T, H), dev)
    if ws is not None:
        w = _want("ws", ws, ws.dtype, ws.shape, dev)
        n = ws.nbytes
    return _check("csa_cache_attn_fwd", LIB.csa_cache_attn_fwd(
        h.ptr, _want("q", q, q.dtype, shape, dev), cmp and cmp._ref, raw and raw._ref, i, k_pad, cc, sk, cu, p0, B, T,
        H, d, ratio, window, softmax_scale, _dtype(q), _want("out", out, q.dtype, shape, dev), ls, w, n,
        _stream_of(h, stream)))
