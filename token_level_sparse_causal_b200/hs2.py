"""Thin ctypes binding over libhs2.so (argument marshalling only).

Every step of the prefill path runs in the library's CUDA kernels; this
module only turns torch tensors into device pointers and sizes, picks the
current CUDA stream, and raises Hs2Error on a non-zero status.  If the shared
library is missing or fails to load, importing the functions raises: there is
no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhs2.so")

(HS2_OK, HS2_ERR_INVALID_ARG, HS2_ERR_UNSUPPORTED, HS2_ERR_WORKSPACE, HS2_ERR_CUDA, HS2_ERR_TIMEOUT, HS2_ERR_INDEX,
 HS2_ERR_RANGE) = range(8)
HS2_KV_BF16, HS2_KV_E4M3 = 0, 1

EXPORTS = ("hs2_full_attn_select", "hs2_sparse_attn", "hs2_sync", "hs2_attn_fwd", "hs2_importance",
           "hs2_topk_select", "hs2_strerror", "hs2_debug_set", "hs2_version", "hs2_launch_count",
           "hs2_full_attn_select_static", "hs2_exp2_check", "hs2_quantize_kv", "hs2_block_select",
           "hs2_full_attn_select_blocks", "hs2_swa_attn", "hs2_sparse_decode",
           "hs2_sparse_decode_workspace", "hs2_attn_fwd_ws", "hs2_qk_norm_rope", "hs2_cache_evict",
           "hs2_varlen_attn", "hs2_tree_attn", "hs2_tree_attn_workspace", "hs2_cache_weights")


class Hs2Shape(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("block", ctypes.c_int32), ("topk", ctypes.c_int32), ("recent", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("q_tok_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("kv_tok_stride", ctypes.c_int64), ("kv_head_stride", ctypes.c_int64)]


class Hs2Cache(ctypes.Structure):
    """hs2_cache: a paged K/V cache (make_cache builds it and keeps its tensors alive)."""
    _fields_ = [("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("page", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("reserved", ctypes.c_int32), ("tok_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p)]


class Hs2Rope(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("Hq", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q_tok_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("kv_tok_stride", ctypes.c_int64), ("kv_head_stride", ctypes.c_int64),
                ("out_tok_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64)]


class Hs2Varlen(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
                ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("q_tok_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("kv_tok_stride", ctypes.c_int64), ("kv_head_stride", ctypes.c_int64)]


class Hs2Draft(ctypes.Structure):
    """hs2_draft: a batch of drafted tokens (make_draft builds it and keeps its tensors alive)."""
    _fields_ = [("n_tok", ctypes.c_int32), ("max_draft", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("q_tok_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("cu_draft", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p), ("mask", ctypes.c_void_p)]


class Hs2Error(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: hs2 status {code} ({strerror(code)})")
        self.code = code


_lib: Optional[ctypes.CDLL] = None

_vp, _i32, _i64, _u32, _u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64
_SIGS = {
    "hs2_full_attn_select": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                             ctypes.POINTER(ctypes.c_size_t), _vp, _i32, _i32, _vp],
    "hs2_full_attn_select_static": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "hs2_full_attn_select_blocks": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    ctypes.POINTER(ctypes.c_size_t), _vp],
    "hs2_block_select": [ctypes.POINTER(Hs2Shape), _vp, _i64, _i32, _i32, _vp, _vp, _vp],
    "hs2_sparse_attn": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "hs2_sync": [_vp],
    "hs2_attn_fwd": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "hs2_attn_fwd_ws": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                        ctypes.POINTER(ctypes.c_size_t), _vp],
    "hs2_swa_attn": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _i32, _vp, _vp, _vp],
    "hs2_sparse_decode": [ctypes.POINTER(Hs2Shape), _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                          ctypes.c_size_t, _vp],
    "hs2_sparse_decode_workspace": [ctypes.POINTER(Hs2Shape), _i32, ctypes.POINTER(ctypes.c_size_t)],
    "hs2_importance": [ctypes.POINTER(Hs2Shape), _vp, _vp, _vp, _vp, _i32, _i32, _vp, _i64, _vp],
    "hs2_topk_select": [ctypes.POINTER(Hs2Shape), _vp, _i64, _i32, _i32, _vp, _vp, _vp],
    "hs2_debug_set": [_u64, _u32],
    "hs2_exp2_check": [_vp, _vp, _vp, _vp, _i64, _vp],
    "hs2_quantize_kv": [_i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp],
    "hs2_version": [],
    "hs2_qk_norm_rope": [ctypes.POINTER(Hs2Cache), ctypes.POINTER(Hs2Rope), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                         _vp, _vp],
    "hs2_cache_evict": [ctypes.POINTER(Hs2Cache), _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp],
    "hs2_varlen_attn": [ctypes.POINTER(Hs2Varlen), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "hs2_tree_attn": [ctypes.POINTER(Hs2Cache), ctypes.POINTER(Hs2Draft), _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "hs2_tree_attn_workspace": [ctypes.POINTER(Hs2Cache), ctypes.POINTER(Hs2Draft), ctypes.POINTER(ctypes.c_size_t)],
    "hs2_cache_weights": [ctypes.POINTER(Hs2Cache), ctypes.POINTER(Hs2Draft), _vp, _vp, _vp, _vp, _i64, _vp],
}


def lib() -> ctypes.CDLL:
    """Load libhs2.so (built in-tree by token_level_sparse_causal_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libhs2.so not built at {LIB_PATH}; run token_level_sparse_causal_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.hs2_launch_count.argtypes = []
        L.hs2_launch_count.restype = ctypes.c_uint64
        L.hs2_strerror.argtypes = [ctypes.c_int]
        L.hs2_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().hs2_strerror(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != HS2_OK:
        raise Hs2Error(rc, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_shape(q: torch.Tensor, k: torch.Tensor, topk: int = 1024, recent: int = 128, block: int = 64,
               kv_dtype: int = HS2_KV_BF16) -> Hs2Shape:
    """hs2_shape for Q [L][Hq][d] and K [L][Hkv][d] tensors (element strides)."""
    L, Hq, d = q.shape
    return Hs2Shape(L=L, Hq=Hq, Hkv=k.shape[1], d=d, block=block, topk=topk, recent=recent, kv_dtype=kv_dtype,
                    q_tok_stride=q.stride(0), q_head_stride=q.stride(1), kv_tok_stride=k.stride(0),
                    kv_head_stride=k.stride(1))


def workspace_bytes(shape: Hs2Shape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().hs2_full_attn_select(ctypes.byref(shape), None, None, None, None, None, None, None, None, None,
                                      None, ctypes.byref(n), None, 0, 0, None), "hs2_full_attn_select(size query)")
    return int(n.value)


def importance_row_stride(shape, b1: int) -> int:
    """Row stride (floats) of hs2_full_attn_select's importance export for the
    block range ending at b1: max(64, roundup(e_{b1-1} - recent, 64))."""
    n_c = max(0, min(shape.L, shape.block * b1) - shape.recent)
    return max(64, (n_c + 63) // 64 * 64)


def hs2_full_attn_select(shape, q, k, v, k_scale, v_scale, o, lse, idx, cnt, workspace, stream=None,
                         importance_out=None, strip=(0, 0)) -> None:
    """importance_out: optional fp32 tensor of Hkv * (b1 - b0) * importance_row_stride(shape, b1)
    elements receiving the importance rows of blocks strip = (b0, b1) that the selection consumed."""
    n = ctypes.c_size_t(workspace.numel() * workspace.element_size())
    _check(lib().hs2_full_attn_select(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale),
                                      _ptr(o), _ptr(lse), _ptr(idx), _ptr(cnt), _ptr(workspace), ctypes.byref(n),
                                      _ptr(importance_out), int(strip[0]), int(strip[1]), _stream(stream)),
           "hs2_full_attn_select")


def hs2_full_attn_select_static(shape, q, k, v, k_scale, v_scale, o, lse, idx, cnt, stream=None) -> None:
    """Same as hs2_full_attn_select, scratch taken from the library's fixed
    16 MiB device array (for callers that cannot allocate)."""
    _check(lib().hs2_full_attn_select_static(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale),
                                             _ptr(v_scale), _ptr(o), _ptr(lse), _ptr(idx), _ptr(cnt),
                                             _stream(stream)), "hs2_full_attn_select_static")


def hs2_full_attn_select_blocks(shape, q, k, v, k_scale, v_scale, o, lse, idx, cnt, workspace, stream=None) -> None:
    n = ctypes.c_size_t(workspace.numel() * workspace.element_size())
    _check(lib().hs2_full_attn_select_blocks(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale),
                                             _ptr(v_scale), _ptr(o), _ptr(lse), _ptr(idx), _ptr(cnt), _ptr(workspace),
                                             ctypes.byref(n), _stream(stream)), "hs2_full_attn_select_blocks")


def hs2_block_select(shape, imp, row_stride, b0, b1, idx, cnt, stream=None) -> None:
    _check(lib().hs2_block_select(ctypes.byref(shape), _ptr(imp), int(row_stride), int(b0), int(b1), _ptr(idx),
                                  _ptr(cnt), _stream(stream)), "hs2_block_select")


def hs2_sparse_attn(shape, q, k, v, k_scale, v_scale, idx, cnt, o, stream=None) -> None:
    _check(lib().hs2_sparse_attn(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale),
                                 _ptr(idx), _ptr(cnt), _ptr(o), _stream(stream)), "hs2_sparse_attn")


def hs2_attn_fwd(shape, q, k, v, k_scale, v_scale, o, lse, stream=None) -> None:
    _check(lib().hs2_attn_fwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale),
                              _ptr(o), _ptr(lse), _stream(stream)), "hs2_attn_fwd")


def attn_fwd_workspace_bytes(shape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().hs2_attn_fwd_ws(ctypes.byref(shape), None, None, None, None, None, None, None, None,
                                 ctypes.byref(n), None), "hs2_attn_fwd_ws(size query)")
    return int(n.value)


def hs2_attn_fwd_ws(shape, q, k, v, k_scale, v_scale, o, lse, workspace, stream=None) -> None:
    """Kernel (1) as the full layer runs it.  A null workspace pointer is the
    C call's size query, so without a workspace this is hs2_attn_fwd."""
    if workspace is None or workspace.numel() == 0:
        hs2_attn_fwd(shape, q, k, v, k_scale, v_scale, o, lse, stream)
        return
    n = ctypes.c_size_t(workspace.numel() * workspace.element_size())
    _check(lib().hs2_attn_fwd_ws(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale),
                                 _ptr(o), _ptr(lse), _ptr(workspace), ctypes.byref(n), _stream(stream)),
           "hs2_attn_fwd_ws")


def sparse_decode_workspace_bytes(shape, n: int) -> int:
    nbytes = ctypes.c_size_t(0)
    _check(lib().hs2_sparse_decode_workspace(ctypes.byref(shape), int(n), ctypes.byref(nbytes)),
           "hs2_sparse_decode_workspace")
    return int(nbytes.value)


def hs2_sparse_decode(shape, q, positions, k, v, k_scale, v_scale, idx, cnt, o, workspace=None,
                      stream=None) -> None:
    """q / o [n][Hq][d] with the strides in `shape`; positions int32 [n] on the device."""
    n = int(positions.numel())
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().hs2_sparse_decode(ctypes.byref(shape), _ptr(q), _ptr(positions), n, _ptr(k), _ptr(v),
                                   _ptr(k_scale), _ptr(v_scale), _ptr(idx), _ptr(cnt), _ptr(o), _ptr(workspace),
                                   nbytes, _stream(stream)), "hs2_sparse_decode")


def hs2_swa_attn(shape, q, k, v, window, o, lse=None, stream=None) -> None:
    _check(lib().hs2_swa_attn(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), int(window), _ptr(o), _ptr(lse),
                              _stream(stream)), "hs2_swa_attn")


def hs2_importance(shape, q, k, k_scale, lse, b0, b1, imp, row_stride, stream=None) -> None:
    _check(lib().hs2_importance(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(k_scale), _ptr(lse), int(b0), int(b1),
                                _ptr(imp), int(row_stride), _stream(stream)), "hs2_importance")


def hs2_topk_select(shape, imp, row_stride, b0, b1, idx, cnt, stream=None) -> None:
    _check(lib().hs2_topk_select(ctypes.byref(shape), _ptr(imp), int(row_stride), int(b0), int(b1), _ptr(idx),
                                 _ptr(cnt), _stream(stream)), "hs2_topk_select")


def hs2_quantize_kv(src, dst, scale, stream=None) -> None:
    """bf16 [L][Hkv][128] -> e4m3 codes (uint8, same shape) + fp32 scales [L][Hkv]."""
    L, Hkv, _ = src.shape
    _check(lib().hs2_quantize_kv(int(L), int(Hkv), _ptr(src), src.stride(0), src.stride(1), _ptr(dst), dst.stride(0),
                                 dst.stride(1), _ptr(scale), _stream(stream)), "hs2_quantize_kv")


def hs2_sync(stream=None) -> None:
    _check(lib().hs2_sync(_stream(stream)), "hs2_sync")


def hs2_launch_count() -> int:
    return int(lib().hs2_launch_count())


def hs2_exp2_check(x, y_mufu, y_fma3, y_fma4, stream=None) -> None:
    _check(lib().hs2_exp2_check(_ptr(x), _ptr(y_mufu), _ptr(y_fma3), _ptr(y_fma4), x.numel(), _stream(stream)),
           "hs2_exp2_check")


# --------------------------------------------- serving around a paged cache --

def _need(t: Optional[torch.Tensor], dtype, shape, what: str, contiguous: bool = True, device: int = None) -> None:
    """Argument check of a device tensor (None passes); `device` is a CUDA device index.  One cheap pass when all is
    well: a decode step makes a dozen of these."""
    if t is None:
        return
    if (t.dtype is not dtype or t.shape != shape or (device is not None and t.get_device() != device)
            or not (t.is_contiguous() if contiguous else t.stride(-1) == 1 or t.shape[-1] == 1)):
        _need_slow(t, dtype, shape, what, contiguous, device)


def _need_slow(t, dtype, shape, what, contiguous=True, device=None) -> None:
    """_need with alternatives: a tuple of dtypes, and None for a free entry of the shape."""
    if t is None:
        return
    ok = t.dtype in (dtype if isinstance(dtype, tuple) else (dtype,)) and t.dim() == len(shape)
    if not ok or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{what}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if not contiguous and t.shape[-1] != 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{what}: on {t.device}, expected device {device}")


def _strides(t: torch.Tensor) -> tuple:
    """Token and head stride of a [tokens][H][d] tensor, with the packed value for a dimension of size 1 (whose
    stride torch leaves open)."""
    (n, H, d), s = t.shape, t.stride()
    head = s[1] if H > 1 else d
    return (s[0] if n > 1 else H * head), head


def _rows(t: torch.Tensor, n: int, H: int, what: str, device: int) -> tuple:
    """Type, shape and device of a bf16 [n][H][128] tensor whose last dimension is contiguous (the library checks the
    other strides); returns its token and head strides (see _strides)."""
    s = t.stride()
    if t.dtype is not torch.bfloat16 or t.shape != (n, H, 128) or s[2] != 1 or t.get_device() != device:
        _need_slow(t, torch.bfloat16, (n, H, 128), what, False, device)
    if n > 1 and H > 1:
        return s[0], s[1]
    return _strides(t)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(name: str, device: int, stream, *args) -> None:
    """Call a library function whose last argument is the stream, on CUDA device `device` (its current stream unless
    one is given)."""
    if device < 0:
        raise ValueError(f"{name}: the tensors must be on a CUDA device")
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(name, device, stream, *args)
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(device)
    else:
        st = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    rc = getattr(_lib or lib(), name)(*args, st)
    if rc != HS2_OK:
        raise Hs2Error(rc, name)


def make_cache(k, v, page_table, page: int, k_scale=None, v_scale=None) -> Hs2Cache:
    """hs2_cache over the pools k, v [n_pages * page][Hkv][128] (bf16; uint8 or
    float8_e4m3fn with fp32 scales [n_pages * page][Hkv]) and an int32 page
    table [n_seqs][max_pages] (None where only hs2_qk_norm_rope uses it)."""
    f8 = k.dtype in (torch.uint8, torch.float8_e4m3fn)
    dev = k.get_device()
    _need_slow(k, (torch.uint8, torch.float8_e4m3fn) if f8 else torch.bfloat16, (None, None, 128), "k", False)
    _need(v, k.dtype, k.shape, "v", False, dev)
    if _strides(v) != _strides(k):
        raise ValueError("v: must have k's strides")
    if page <= 0 or k.shape[0] % page:
        raise ValueError(f"page: {page} does not divide the pools' {k.shape[0]} tokens")
    if f8 != (k_scale is not None) or f8 != (v_scale is not None):
        raise ValueError("k_scale, v_scale: given exactly with an e4m3 cache")
    _need(k_scale, torch.float32, (k.shape[0], k.shape[1]), "k_scale", True, dev)
    _need(v_scale, torch.float32, (k.shape[0], k.shape[1]), "v_scale", True, dev)
    _need_slow(page_table, torch.int32, (None, None), "page_table", True, dev)
    n_seqs, max_pages = (0, 0) if page_table is None else page_table.shape
    c = Hs2Cache(Hkv=k.shape[1], d=k.shape[2], kv_dtype=HS2_KV_E4M3 if f8 else HS2_KV_BF16, page=page,
                 n_pages=k.shape[0] // page, n_seqs=n_seqs, max_pages=max_pages, tok_stride=_strides(k)[0],
                 head_stride=_strides(k)[1], k=_addr(k), v=_addr(v), k_scale=_addr(k_scale), v_scale=_addr(v_scale),
                 page_table=_addr(page_table))
    c.tensors, c.device = (k, v, page_table, k_scale, v_scale), dev
    return c


def hs2_qk_norm_rope(cache: Hs2Cache, q, k, v, q_weight, k_weight, eps: float, inv_freq, positions, slots, q_out,
                     interleaved: bool = False, stream=None) -> None:
    """q, q_out [n][Hq][128], k, v [n][Hkv][128] bf16, inv_freq float64 [rot / 2], positions and slots int32 [n] (slots
    None: rows 0 .. n - 1 of the pools; -1: no cache write).  Strides are multiples of 8, a head's 128 at least; q's
    and q_out's heads lie within their token (heads outermost is refused)."""
    n, Hq, _ = q.shape
    dev, Hkv, rot = cache.device, cache.Hkv, 2 * inv_freq.numel()
    qs, outs = _rows(q, n, Hq, "q", dev), _rows(q_out, n, Hq, "q_out", dev)
    kv = _rows(k, n, Hkv, "k", dev)
    if _rows(v, n, Hkv, "v", dev) != kv:
        raise ValueError("v: must have k's strides")
    _need(q_weight, torch.bfloat16, (128,), "q_weight", True, dev)
    _need(k_weight, torch.bfloat16, (128,), "k_weight", True, dev)
    _need(inv_freq, torch.float64, (rot // 2,), "inv_freq", True, dev)
    _need(positions, torch.int32, (n,), "positions", True, dev)
    _need(slots, torch.int32, (n,), "slots", True, dev)
    if slots is None and n > cache.n_pages * cache.page:
        raise ValueError(f"slots: {n} rows do not fit the pools' {cache.n_pages * cache.page} tokens")
    r = Hs2Rope(n, Hq, rot, 1 if interleaved else 0, eps, 0, qs[0], qs[1], kv[0], kv[1], outs[0], outs[1])
    _call("hs2_qk_norm_rope", dev, stream, ctypes.byref(cache), ctypes.byref(r), q.data_ptr(), k.data_ptr(),
          v.data_ptr(), _addr(q_weight), _addr(k_weight), inv_freq.data_ptr(), positions.data_ptr(), _addr(slots),
          q_out.data_ptr())


def make_varlen(q, k, n_seqs: int) -> Hs2Varlen:
    """hs2_varlen for packed q [total_q][Hq][128] and k (v alike) [total_k][Hkv][128], bf16."""
    _need_slow(q, torch.bfloat16, (None, None, 128), "q", False)
    _need_slow(k, torch.bfloat16, (None, None, 128), "k", False, q.get_device())
    return Hs2Varlen(n_seqs, q.shape[0], k.shape[0], q.shape[1], k.shape[1], 128, *_strides(q), *_strides(k))


def hs2_varlen_attn(shape: Hs2Varlen, q, k, v, cu_q, cu_k, o, lse=None, stream=None) -> None:
    """q, o [total_q][Hq][128], k, v [total_k][Hkv][128]; cu_q, cu_k int32 [n_seqs + 1] (cu_k None: cu_q);
    lse fp32 [Hq][total_q] or None.  q and o, and k and v, have the strides make_varlen saw."""
    dev = q.get_device()
    st_q, st_k = (shape.q_tok_stride, shape.q_head_stride), (shape.kv_tok_stride, shape.kv_head_stride)
    for t, n, H, st, name in ((q, shape.total_q, shape.Hq, st_q, "q"), (o, shape.total_q, shape.Hq, st_q, "o"),
                              (k, shape.total_k, shape.Hkv, st_k, "k"), (v, shape.total_k, shape.Hkv, st_k, "v")):
        found = _rows(t, n, H, name, dev)
        if found != st:
            raise ValueError(f"{name}: strides {found}, expected {st}")
    _need(cu_q, torch.int32, (shape.n_seqs + 1,), "cu_q", True, dev)
    _need(cu_k, torch.int32, (shape.n_seqs + 1,), "cu_k", True, dev)
    _need(lse, torch.float32, (shape.Hq, shape.total_q), "lse", True, dev)
    _call("hs2_varlen_attn", dev, stream, ctypes.byref(shape), _addr(q), _addr(k), _addr(v), _addr(cu_q), _addr(cu_k),
          _addr(o), _addr(lse))


def make_draft(q, cu_draft, ctx_len, mask, max_draft: int) -> Hs2Draft:
    """hs2_draft for queries shaped like q [n_tok][Hq][128]; cu_draft int32 [n_seqs + 1], ctx_len int32 [n_seqs],
    mask int64 or uint64 [n_tok] (None: chains)."""
    dev = q.get_device()
    _need_slow(q, torch.bfloat16, (None, None, 128), "q", False)
    _need_slow(ctx_len, torch.int32, (None,), "ctx_len", True, dev)
    _need(cu_draft, torch.int32, (ctx_len.shape[0] + 1,), "cu_draft", True, dev)
    _need_slow(mask, (torch.int64, torch.uint64), (q.shape[0],), "mask", True, dev)
    d = Hs2Draft(q.shape[0], int(max_draft), q.shape[1], 0, *_strides(q), _addr(cu_draft), _addr(ctx_len), _addr(mask))
    d.tensors, d.n_seqs, d.device = (cu_draft, ctx_len, mask), ctx_len.shape[0], dev
    return d


def _need_draft(cache: Hs2Cache, draft: Hs2Draft, q, o=None) -> None:
    if draft.n_seqs != cache.n_seqs:
        raise ValueError(f"draft: {draft.n_seqs} sequences, the cache has {cache.n_seqs}")
    if draft.device != cache.device:
        raise ValueError(f"draft: on device {draft.device}, the cache is on {cache.device}")
    st = (draft.q_tok_stride, draft.q_head_stride)
    for t, name in ((q, "q"), (o, "o")):
        if t is not None and _rows(t, draft.n_tok, draft.Hq, name, cache.device) != st:
            raise ValueError(f"{name}: strides {_strides(t)}, the draft's are {st}")


def tree_attn_workspace_bytes(cache: Hs2Cache, draft: Hs2Draft) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().hs2_tree_attn_workspace(ctypes.byref(cache), ctypes.byref(draft), ctypes.byref(n)),
           "hs2_tree_attn_workspace")
    return int(n.value)


def hs2_tree_attn(cache: Hs2Cache, draft: Hs2Draft, q, o, lse, workspace, stream=None) -> None:
    """q, o [n_tok][Hq][128] bf16; lse fp32 [Hq][n_tok] or None; workspace of tree_attn_workspace_bytes."""
    _need_draft(cache, draft, q, o)
    _need(lse, torch.float32, (draft.Hq, draft.n_tok), "lse", True, cache.device)
    if workspace.get_device() != cache.device:
        raise ValueError(f"workspace: on {workspace.device}, expected device {cache.device}")
    _call("hs2_tree_attn", cache.device, stream, ctypes.byref(cache), ctypes.byref(draft), _addr(q), _addr(o),
          _addr(lse), _addr(workspace), workspace.numel() * workspace.element_size())


def hs2_cache_weights(cache: Hs2Cache, draft: Hs2Draft, q, lse, counted, acc, stream=None) -> None:
    """lse fp32 [Hq][n_tok] from hs2_tree_attn; counted uint8 [n_tok] or None; acc fp32 [n_seqs][Hkv][acc_stride]."""
    _need_draft(cache, draft, q)
    _need(lse, torch.float32, (draft.Hq, draft.n_tok), "lse", True, cache.device)
    _need_slow(counted, (torch.uint8, torch.bool), (draft.n_tok,), "counted", True, cache.device)
    _need(acc, torch.float32, (cache.n_seqs, cache.Hkv, acc.shape[-1]), "acc", True, cache.device)
    _call("hs2_cache_weights", cache.device, stream, ctypes.byref(cache), ctypes.byref(draft), _addr(q), _addr(lse),
          _addr(counted), _addr(acc), acc.shape[2])


def hs2_cache_evict(cache: Hs2Cache, seq_len, acc, keep: int, recent: int, idx, new_len, acc_out=None,
                    stream=None) -> None:
    """seq_len, new_len int32 [n_seqs]; acc (and acc_out, which may be acc) fp32 [n_seqs][Hkv][acc_stride];
    idx int32 [n_seqs][Hkv][keep]."""
    dev, B = cache.device, cache.n_seqs
    _need(seq_len, torch.int32, (B,), "seq_len", True, dev)
    _need(new_len, torch.int32, (B,), "new_len", True, dev)
    _need(acc, torch.float32, (B, cache.Hkv, acc.shape[-1]), "acc", True, dev)
    _need(acc_out, torch.float32, acc.shape, "acc_out", True, dev)
    _need(idx, torch.int32, (B, cache.Hkv, keep), "idx", True, dev)
    _call("hs2_cache_evict", dev, stream, ctypes.byref(cache), _addr(seq_len), _addr(acc), _addr(acc_out),
          acc.shape[2], int(keep), int(recent), _addr(idx), _addr(new_len))


# hs2_debug_set flag bits (include/hs2.h)
DEBUG_SKIP_LOADS, DEBUG_IMP_VISIBLE, DEBUG_FA_CTA_PAIRS, DEBUG_FAIL_TMAP = 1, 2, 4, 8


def hs2_debug_set(wait_limit_ns: int = 2_000_000_000, flags: int = 0) -> None:
    _check(lib().hs2_debug_set(int(wait_limit_ns), int(flags)), "hs2_debug_set")


# ------------------------------------------------------------ conveniences --

def alloc_outputs(shape: Hs2Shape, q: torch.Tensor, with_workspace: bool = True) -> dict:
    """Device buffers for one full-layer call (torch supplies the memory)."""
    dev = q.device
    nb = shape.L // shape.block
    out = {
        "o": torch.empty_like(q),
        "lse": torch.empty((shape.Hq, shape.L), device=dev, dtype=torch.float32),
        "idx": torch.empty((shape.Hkv, nb, shape.topk + shape.recent), device=dev, dtype=torch.int32),
        "cnt": torch.empty((shape.Hkv, nb), device=dev, dtype=torch.int32),
    }
    if with_workspace:
        out["workspace"] = torch.empty(workspace_bytes(shape) // 4 + 4, device=dev, dtype=torch.float32)
    return out
