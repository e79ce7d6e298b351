"""ctypes binding of ``libgdn_b200.so`` (declared in ``include/gdn.h``).

Argument marshalling only: torch tensors become device pointers, sizes and
the current CUDA stream; every step of the computation runs in the library's
kernels. There is no CPU fallback: if the library is missing or a tensor is
not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_DEBUG_CHECKS=1 in the environment selects the index-checking build (see build.py --debug)
_LIB_PATH = os.path.join(_HERE, "libgdn_b200_debug.so" if os.environ.get("GDN_DEBUG_CHECKS") == "1"
                         else "libgdn_b200.so")
_lib = None

GDN_F32, GDN_BF16 = 0, 1
_DTYPE = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
STATUS = {0: "GDN_OK", 1: "GDN_ERR_NULL", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_DTYPE", 4: "GDN_ERR_ALIGN",
          5: "GDN_ERR_SEQLENS", 6: "GDN_ERR_WORKSPACE", 7: "GDN_ERR_CUDA", 8: "GDN_ERR_TIMEOUT",
          9: "GDN_ERR_BOUNDS", 10: "GDN_ERR_PAGES"}

# Every symbol include/gdn.h declares, with its ctypes signature.
_VP, _SZ, _I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_I64, _F32, _F64 = ctypes.c_int64, ctypes.c_float, ctypes.c_double
SIGNATURES = {
    "gdn_version": (_I, []),
    "gdn_last_error": (ctypes.c_char_p, []),
    "gdn_chunk_fwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "gdn_chunk_fwd": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _SZ, _VP]),
    "gdn_chunk_fwd_raw": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _SZ, _VP]),
    "gdn_decode_step_raw": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP]),
    "gdn_chunk_fwd_check": (_I, [_VP, _SZ, _VP]),
    "gdn_attn_fwd": (_I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, ctypes.c_float, _I, _VP, _VP, _SZ, _VP]),
    "gdn_qk_norm_rope": (_I, [_VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _F32, _VP, _I, _I, _I, _I, _I, _F64, _I, _VP,
                              _VP, _VP, _VP, _VP, _I, _I, _VP, _SZ, _VP]),
    "gdn_attn_prefill": (_I, [_VP, _I64, _VP, _I64, _VP, _I64, _VP, _I, _I, _I, _I, _I, _I, _F32, _I, _VP, _VP, _SZ,
                              _VP]),
    "gdn_attn_decode_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "gdn_attn_decode": (_I, [_VP, _VP, _VP, _I, _I, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _F32, _I, _VP, _VP, _SZ, _VP]),
    "gdn_proj_w8": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "gdn_decode_step": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP]),
    "gdn_seq_scan": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP, _VP, _VP]),
    "gdn_diag_mma_tile": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP]),
    "gdn_diag_ut_solve": (_I, [_VP, _VP, _VP]),
    "gdn_chunk_fwd_noalloc": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP, _VP, _VP]),
    "gdn_debug_inject": (_I, [_I, ctypes.c_uint]),
    "gdn_profile_enable": (None, [_I]),
    "gdn_profile_read": (_I, [ctypes.c_char_p, _SZ, _VP, _VP, _I]),
}


class GdnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (STATUS.get(status, str(status)), msg))
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load (once) and return the ctypes handle; raises if the library was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise GdnError(-1, "CUDA library %s not built (run python -m "
                           "linear_attention_recurrent_chunked_b200.build)" % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status: int):
    if status != 0:
        raise GdnError(status, load_library().gdn_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise GdnError(1, "tensors must be on a CUDA device (no CPU path)")
            if not t.is_contiguous():
                raise GdnError(2, "tensors must be contiguous")


def chunk_fwd_workspace_size(N: int, T_tot: int, H: int, dk: int, dv: int, dtype: torch.dtype) -> int:
    return int(load_library().gdn_chunk_fwd_workspace_size(N, T_tot, H, dk, dv, _DTYPE[dtype]))


_cached = threading.local()  # each thread's workspaces, which end with it


def _bytes(n, index):
    return torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", index))


def _stream_and_ws(index, nbytes, workspace):
    """The current stream of a device, and a workspace: the caller's, or the cached one of this device, stream
    and thread (the kernels of two threads' calls on one stream may take turns), or while a graph is being captured a
    fresh one, so that the graph keeps memory of its own."""
    stream = torch._C._cuda_getCurrentRawStream(index)
    if workspace is None:
        if torch._C._cuda_isCurrentStreamCapturing():
            workspace = _bytes(max(nbytes, 256), index)
        else:
            mine, key = _cached.__dict__, (index, stream)
            workspace = mine.get(key)
            if workspace is None or workspace.numel() < nbytes:
                workspace = mine[key] = _bytes(max(nbytes, 256), index)
        return stream, workspace, workspace.numel()
    if not workspace.is_contiguous() or workspace.get_device() != index:
        raise GdnError(6, "workspace must be a contiguous tensor on the inputs' device")
    return stream, workspace, workspace.numel() * workspace.element_size()


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NOTHING = _Nothing()


def _on(index):
    """Makes the tensors' device the current one for a call, where it is not."""
    return _NOTHING if index == torch._C._cuda_getDevice() else torch.cuda.device(index)


def chunk_fwd(q, k, v, g, beta, S0=None, cu_seqlens=None, N: Optional[int] = None, o=None, S_T=None,
              workspace=None, check: bool = False):
    """Chunked prefill. q,k [T,H,dk], v [T,H,dv] (fp32 or bf16); g,beta [T,H] fp32;
    S0 [N,H,dv,dk] fp32 or None; cu_seqlens [N+1] int32 (device) or None (then N
    equal sequences, N from ``N``, S0, else 1). Returns (o, S_T). With
    check=True the stream is synchronised and the device error word read."""
    lib = load_library()
    _need_cuda(q, k, v, g, beta, S0, cu_seqlens, o, S_T, workspace)
    T_tot, H, dk = q.shape
    dv = v.shape[2]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    elif N is None:
        N = S0.shape[0] if S0 is not None else 1
    if o is None:
        o = torch.empty((T_tot, H, dv), dtype=q.dtype, device=q.device)
    if S_T is None:
        S_T = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    dt = _DTYPE.get(q.dtype, 99)
    need = int(lib.gdn_chunk_fwd_workspace_size(N, T_tot, H, dk, dv, dt))
    index = q.get_device()
    with _on(index):
        stream, ws, ws_bytes = _stream_and_ws(index, need, workspace)
        _check(lib.gdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
                                 N, T_tot, H, dk, dv, dt, _ptr(o), _ptr(S_T), ws.data_ptr(), ws_bytes, stream))
        if check:
            _check(lib.gdn_chunk_fwd_check(ws.data_ptr(), ws_bytes, stream))
    return o, S_T


def chunk_fwd_raw(q_raw, k_raw, v, a, b, S0=None, cu_seqlens=None, N: Optional[int] = None, o=None, S_T=None,
                  workspace=None, check: bool = False):
    """Chunked prefill from raw inputs (see include/gdn.h): q_raw, k_raw [T,H,dk] of any norm,
    v [T,H,dv]; a, b [T,H] fp32 gate logits (g = -softplus(a), beta = sigmoid(b)); the rest as
    chunk_fwd. The normalisation and gates run inside the library's kernels."""
    lib = load_library()
    _need_cuda(q_raw, k_raw, v, a, b, S0, cu_seqlens, o, S_T, workspace)
    T_tot, H, dk = q_raw.shape
    dv = v.shape[2]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    elif N is None:
        N = S0.shape[0] if S0 is not None else 1
    if o is None:
        o = torch.empty((T_tot, H, dv), dtype=q_raw.dtype, device=q_raw.device)
    if S_T is None:
        S_T = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q_raw.device)
    dt = _DTYPE.get(q_raw.dtype, 99)
    need = int(lib.gdn_chunk_fwd_workspace_size(N, T_tot, H, dk, dv, dt))
    index = q_raw.get_device()
    with _on(index):
        stream, ws, ws_bytes = _stream_and_ws(index, need, workspace)
        _check(lib.gdn_chunk_fwd_raw(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(a), _ptr(b), _ptr(S0), _ptr(cu_seqlens),
                                     N, T_tot, H, dk, dv, dt, _ptr(o), _ptr(S_T), ws.data_ptr(), ws_bytes, stream))
        if check:
            _check(lib.gdn_chunk_fwd_check(ws.data_ptr(), ws_bytes, stream))
    return o, S_T


def decode_step_raw(q_raw, k_raw, v, a, b, S, o=None):
    """One decode step from raw inputs (q, k normalised and gates applied in the kernel)."""
    lib = load_library()
    _need_cuda(q_raw, k_raw, v, a, b, S, o)
    B, H, dk = q_raw.shape
    dv = v.shape[2]
    if o is None:
        o = torch.empty((B, H, dv), dtype=q_raw.dtype, device=q_raw.device)
    _check(lib.gdn_decode_step_raw(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(a), _ptr(b), _ptr(S), B, H, dk, dv,
                                   _DTYPE.get(q_raw.dtype, 99), _ptr(o), _stream()))
    return o


def proj_w8(x, w, scale, H: int, dk: int, dv: int, out=None, workspace=None, check: bool = False):
    """Input projection with int8 weights (see include/gdn.h): x [T, D] bf16, w [N, D] int8,
    scale [N] fp32, N = H (2 dk + dv) + 2 H. Returns (q_raw [T,H,dk], k_raw [T,H,dk], v [T,H,dv]
    bf16, a [T,H], b [T,H] fp32); ``out`` may pass those five tensors to write into."""
    lib = load_library()
    _need_cuda(x, w, scale, workspace)
    T, D = x.shape
    dev = x.device
    if out is None:
        out = (torch.empty((T, H, dk), dtype=torch.bfloat16, device=dev),
               torch.empty((T, H, dk), dtype=torch.bfloat16, device=dev),
               torch.empty((T, H, dv), dtype=torch.bfloat16, device=dev),
               torch.empty((T, H), dtype=torch.float32, device=dev),
               torch.empty((T, H), dtype=torch.float32, device=dev))
    _need_cuda(*out)
    index = x.get_device()
    with _on(index):
        stream, ws, ws_bytes = _stream_and_ws(index, 256, workspace)
        _check(lib.gdn_proj_w8(_ptr(x), _ptr(w), _ptr(scale), T, D, H, dk, dv, *[_ptr(t) for t in out], ws.data_ptr(),
                               ws_bytes, stream))
        if check:
            _check(lib.gdn_chunk_fwd_check(ws.data_ptr(), ws_bytes, stream))
    return out


def attn_fwd(q, k, v, cu_seqlens=None, N: Optional[int] = None, max_len: Optional[int] = None,
             scale: float = 0.0, o=None, workspace=None, check: bool = False):
    """Causal attention (see include/gdn.h): q, k, v [T, H, 128] bf16; cu_seqlens [N+1] int32
    (device) or None (N equal sequences, N from ``N``, else 1); max_len bounds the sequence
    lengths (required with cu_seqlens); scale <= 0 means 1 / sqrt(128). Returns o [T, H, 128]."""
    lib = load_library()
    _need_cuda(q, k, v, cu_seqlens, o, workspace)
    T_tot, H, d = q.shape
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        if max_len is None:
            raise GdnError(2, "max_len is required with cu_seqlens")
    else:
        N = 1 if N is None else N
        max_len = T_tot // N
    if o is None:
        o = torch.empty_like(q)
    index = q.get_device()
    with _on(index):
        stream, ws, ws_bytes = _stream_and_ws(index, 256, workspace)
        _check(lib.gdn_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), N, T_tot, H, d, max_len, float(scale),
                                _DTYPE.get(q.dtype, 99), _ptr(o), ws.data_ptr(), ws_bytes, stream))
        if check:
            _check(lib.gdn_chunk_fwd_check(ws.data_ptr(), ws_bytes, stream))
    return o


def _refuse(name, t, index, dtype, shape):
    """Says what is wrong with a tensor that one of the checks below did not accept."""
    if not isinstance(t, torch.Tensor):
        raise GdnError(1, "%s is %r, not a tensor" % (name, type(t).__name__))
    if t.dtype != dtype:
        raise GdnError(3, "%s is %s, not %s" % (name, t.dtype, dtype))
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise GdnError(2, "%s has shape %s, not %s" % (name, tuple(t.shape), tuple("*" if n is None else n for n in shape)))
    if not t.is_cuda or t.get_device() != index:
        raise GdnError(1, "%s is on %s (all tensors must be on one CUDA device; no CPU path)" % (name, t.device))
    raise GdnError(2, "%s must be contiguous%s" % (name, " within a token" if len(shape) == 3 else ""))


def _flat(name, t, index, dtype, shape):
    """Address of a contiguous tensor on device `index` with this type and shape."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _refuse(name, t, index, dtype, shape)


def _heads(name, t, index, dtype, T, H, d):
    """Address and token stride of a [T, H, d] tensor whose tokens are contiguous: a token's heads may be
    a slice of a wider row."""
    if t.dtype is dtype and t.shape == (T, H, d) and t.get_device() == index:
        st, s1, s2 = t.stride()
        if (s2 == 1 and (s1 == d or H == 1)) or not T:
            return t.data_ptr(), st if T > 1 else H * d
    _refuse(name, t, index, dtype, (T, H, d))


def _index(name, t):
    """The device that a call runs on: its first tensor's."""
    if t.dim() != 3 or not t.is_cuda:
        _refuse(name, t, 0, t.dtype, (None, None, None))
    return t.get_device()


_BF16, _I32, _FP32 = torch.bfloat16, torch.int32, torch.float32


def qk_norm_rope(q, k, wq, wk, positions, v=None, rot: Optional[int] = None, base: float = 10000.0, eps: float = 1e-6,
                 q_out=None, k_out=None, k_cache=None, v_cache=None, slots=None, want_k: bool = True, workspace=None,
                 check: bool = False):
    """Norms of queries and keys per head with the position rotation in the same pass (see
    include/gdn.h). q [T,Hq,d], k, v [T,Hkv,d] (fp32 or bf16; may be slices of a fused projection's
    output); wq, wk [d] fp32 or None; positions [T] int32; rot rotated elements (None: all d, 0: none).
    With slots [T] int32 the rotated keys and the values also go to k_cache, v_cache
    [pages,Hkv,page_size,d]. Returns (q_out, k_out); k_out is None with want_k=False, for callers that
    read the keys from the cache."""
    lib = load_library()
    dtype = q.dtype
    if dtype not in _DTYPE:
        raise GdnError(3, "q is %s (float32 or bfloat16)" % dtype)
    index = _index("q", q)
    T, Hq, d = q.shape
    Hkv = k.shape[1] if k.dim() == 3 else -1
    pq, q_stride = _heads("q", q, index, dtype, T, Hq, d)
    pk, k_stride = _heads("k", k, index, dtype, T, Hkv, d)
    pv = pkc = pvc = ps = None
    v_stride = pages = page_size = 0
    if slots is not None:
        if v is None or k_cache is None or v_cache is None:
            raise GdnError(1, "slots needs v, k_cache and v_cache")
        pv, v_stride = _heads("v", v, index, dtype, T, Hkv, d)
        shape = k_cache.shape
        if len(shape) != 4 or shape[1] != Hkv or shape[3] != d:
            _refuse("k_cache", k_cache, index, dtype, (None, Hkv, None, d))
        pages, page_size = shape[0], shape[2]
        pkc = _flat("k_cache", k_cache, index, dtype, shape)
        pvc = _flat("v_cache", v_cache, index, dtype, shape)
        ps = _flat("slots", slots, index, _I32, (T,))
    elif k_cache is not None or v_cache is not None:
        raise GdnError(1, "k_cache and v_cache need slots")
    pwq = None if wq is None else _flat("wq", wq, index, _FP32, (d,))
    pwk = None if wk is None else _flat("wk", wk, index, _FP32, (d,))
    pp = None if positions is None else _flat("positions", positions, index, _I32, (T,))
    with _on(index):
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            pqo = q_out.data_ptr()
        else:
            pqo = _flat("q_out", q_out, index, dtype, (T, Hq, d))
        pko = None
        if k_out is not None:
            pko = _flat("k_out", k_out, index, dtype, (T, Hkv, d))
        elif want_k:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
            pko = k_out.data_ptr()
        stream, ws, ws_bytes = _stream_and_ws(index, 256, workspace)
        _check(lib.gdn_qk_norm_rope(pq, q_stride, pk, k_stride, pv, v_stride, pwq, pwk, eps, pp, T, Hq, Hkv, d,
                                    d if rot is None else rot, base, _DTYPE[dtype], pqo, pko, pkc, pvc, ps, pages, page_size,
                                    ws.data_ptr(), ws_bytes, stream))
        if check:
            _check(lib.gdn_chunk_fwd_check(ws.data_ptr(), ws_bytes, stream))
    return q_out, k_out


def attn_prefill(q, k, v, cu_seqlens=None, N: Optional[int] = None, max_len: Optional[int] = None, scale: float = 0.0,
                 o=None, workspace=None, check: bool = False):
    """Causal attention over whole prompts with grouped heads (see include/gdn.h): q [T,Hq,d], k, v
    [T,Hkv,d] bf16 (d 64 or 128; may be slices of wider rows); cu_seqlens [N+1] int32 (device) or None
    (N equal sequences, N from ``N``, else 1); max_len bounds the lengths (required with cu_seqlens);
    scale <= 0 means 1 / sqrt(d). Returns o [T,Hq,d]."""
    lib = load_library()
    if q.dtype is not _BF16:
        raise GdnError(3, "q is %s, not %s" % (q.dtype, _BF16))
    index = _index("q", q)
    T, Hq, d = q.shape
    Hkv = k.shape[1] if k.dim() == 3 else -1
    pq, q_stride = _heads("q", q, index, _BF16, T, Hq, d)
    pk, k_stride = _heads("k", k, index, _BF16, T, Hkv, d)
    pv, v_stride = _heads("v", v, index, _BF16, T, Hkv, d)
    pcu = None
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        pcu = _flat("cu_seqlens", cu_seqlens, index, _I32, (N + 1,))
        if max_len is None:
            raise GdnError(2, "max_len is required with cu_seqlens")
        max_len = min(max_len, T)
    else:
        N = 1 if N is None else N
        if N < 1:
            raise GdnError(2, "N=%d must be >= 1" % N)
        max_len = T // N
    with _on(index):
        if o is None:
            o = torch.empty_like(q, memory_format=torch.contiguous_format)
            po = o.data_ptr()
        else:
            po = _flat("o", o, index, _BF16, (T, Hq, d))
        stream, ws, ws_bytes = _stream_and_ws(index, 256, workspace)
        _check(lib.gdn_attn_prefill(pq, q_stride, pk, k_stride, pv, v_stride, pcu, N, T, Hq, Hkv, d, max_len, scale, GDN_BF16,
                                    po, ws.data_ptr(), ws_bytes, stream))
        if check:
            _check(lib.gdn_chunk_fwd_check(ws.data_ptr(), ws_bytes, stream))
    return o


def attn_decode(q, k_cache, v_cache, page_table, lens, prefix_pages=None, prefix_len: int = 0, scale: float = 0.0, o=None,
                workspace=None, check: bool = False):
    """Attention of one new token per sequence over the paged cache (see include/gdn.h): q [B,Hq,d]
    bf16, k_cache, v_cache [pages,Hkv,page_size,d] bf16, page_table [B,max_pages] int32, lens [B] int32;
    prefix_pages [n] int32 and prefix_len: a prefix that all sequences share. B and max_pages may be 0 here.
    Returns o [B,Hq,d]."""
    lib = load_library()
    if q.dtype is not _BF16:
        raise GdnError(3, "q is %s, not %s" % (q.dtype, _BF16))
    shape, table = k_cache.shape, page_table.shape
    B, Hq, d = q.shape if q.dim() == 3 else (-1, -1, -1)
    if len(shape) != 4 or shape[3] != d:
        _refuse("k_cache", k_cache, 0, _BF16, (None, None, None, d))
    if len(table) != 2:
        _refuse("page_table", page_table, 0, _I32, (B, None))
    pages, Hkv, page_size, _ = shape
    if v_cache.shape != shape:
        _refuse("v_cache", v_cache, 0, _BF16, shape)
    if lens.shape != (B,):
        _refuse("lens", lens, 0, _I32, (B,))
    if page_table.dtype is not _I32:
        _refuse("page_table", page_table, 0, _I32, (B, None))
    if prefix_len:
        if prefix_pages is None:
            raise GdnError(1, "prefix_len needs prefix_pages")
        if prefix_len > prefix_pages.numel() * page_size:
            raise GdnError(2, "prefix_len=%d exceeds the %d prefix pages" % (prefix_len, prefix_pages.numel()))
    if not q.is_contiguous():
        raise GdnError(2, "q must be contiguous")
    index = _index("q", q)
    pq = _flat("q", q, index, _BF16, (B, Hq, d))
    pk = _flat("k_cache", k_cache, index, _BF16, shape)
    pv = _flat("v_cache", v_cache, index, _BF16, shape)
    pt = _flat("page_table", page_table, index, _I32, (B, table[1]))
    pl = _flat("lens", lens, index, _I32, (B,))
    pp = _flat("prefix_pages", prefix_pages, index, _I32, (prefix_pages.numel(),)) if prefix_len else None
    with _on(index):
        if o is None:
            o = torch.empty_like(q)
            po = o.data_ptr()
        else:
            po = _flat("o", o, index, _BF16, (B, Hq, d))
        if not B:
            return o
        columns = table[1]
        if not columns:  # the library wants one: of no page
            page_table, columns = page_table.new_full((B, 1), -1), 1
            pt = page_table.data_ptr()
        stream, ws, ws_bytes = _stream_and_ws(index, lib.gdn_attn_decode_workspace_size(B, Hq, Hkv, d, prefix_len), workspace)
        _check(lib.gdn_attn_decode(pq, pk, pv, pages, page_size, pt, columns, pl, pp, prefix_len, B, Hq, Hkv, d, scale,
                                   GDN_BF16, po, ws.data_ptr(), ws_bytes, stream))
        if check:
            _check(lib.gdn_chunk_fwd_check(ws.data_ptr(), ws_bytes, stream))
    return o


def chunk_fwd_noalloc(q, k, v, g, beta, S0=None, cu_seqlens=None, N: Optional[int] = None, o=None, S_T=None):
    """chunk_fwd without a workspace argument: the library's built-in scratch
    array is used instead (see include/gdn.h). o and S_T are allocated here
    only when the caller does not pass them."""
    lib = load_library()
    _need_cuda(q, k, v, g, beta, S0, cu_seqlens, o, S_T)
    T_tot, H, dk = q.shape
    dv = v.shape[2]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    elif N is None:
        N = S0.shape[0] if S0 is not None else 1
    if o is None:
        o = torch.empty((T_tot, H, dv), dtype=q.dtype, device=q.device)
    if S_T is None:
        S_T = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    _check(lib.gdn_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
                                     N, T_tot, H, dk, dv, _DTYPE.get(q.dtype, 99), _ptr(o), _ptr(S_T), _stream()))
    return o, S_T


def decode_step(q, k, v, g, beta, S, o=None):
    """One decode step for B sequences: q,k [B,H,dk], v [B,H,dv], g,beta [B,H],
    S [B,H,dv,dk] fp32 updated in place. Returns o [B,H,dv]."""
    lib = load_library()
    _need_cuda(q, k, v, g, beta, S, o)
    B, H, dk = q.shape
    dv = v.shape[2]
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    _check(lib.gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), B, H, dk, dv,
                               _DTYPE.get(q.dtype, 99), _ptr(o), _stream()))
    return o


def seq_scan(q, k, v, g, beta, S0=None, cu_seqlens=None, N: Optional[int] = None, o=None, S_T=None):
    """Token-by-token scan on the GPU (comparator). Same arguments as chunk_fwd."""
    lib = load_library()
    _need_cuda(q, k, v, g, beta, S0, cu_seqlens, o, S_T)
    T_tot, H, dk = q.shape
    dv = v.shape[2]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    elif N is None:
        N = S0.shape[0] if S0 is not None else 1
    if o is None:
        o = torch.empty((T_tot, H, dv), dtype=q.dtype, device=q.device)
    if S_T is None:
        S_T = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    _check(lib.gdn_seq_scan(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
                            N, T_tot, H, dk, dv, _DTYPE.get(q.dtype, 99), _ptr(o), _ptr(S_T), _stream()))
    return o, S_T


def diag_mma_tile(A, B, a_mn: int = 0, b_mn: int = 0, variant: int = 0):
    """Diagnostic single tensor-core tile: returns the [128, N] TMEM dump of
    A [M,K] @ B [N,K]^T (bf16 in, fp32 out). See include/gdn.h."""
    lib = load_library()
    _need_cuda(A, B)
    M, K = A.shape
    N = B.shape[0]
    D = torch.full((128, N), float("nan"), dtype=torch.float32, device=A.device)
    _check(lib.gdn_diag_mma_tile(_ptr(A), _ptr(B), _ptr(D), M, N, K, a_mn, b_mn, variant, _stream()))
    return D


def debug_inject(kind: int, wait_us: int = 0) -> None:
    """Failure injection for tests (see include/gdn.h): 0 = off, 1 = withhold the first
    segment's end state of head 0 so that the blocks waiting for it time out after wait_us; 2, 3 =
    withhold a load of keys or values in the attention layer's kernels likewise."""
    _check(load_library().gdn_debug_inject(kind, wait_us))


def profile_enable(on: bool = True) -> None:
    """Record CUDA events around every kernel the library launches (see include/gdn.h)."""
    load_library().gdn_profile_enable(1 if on else 0)


def profile_read() -> dict:
    """{kernel name: (total ms, launches)} since the last read; waits for the recorded events."""
    lib = load_library()
    n_max = 64
    names = ctypes.create_string_buffer(8192)
    ms = (ctypes.c_float * n_max)()
    cnt = (ctypes.c_int * n_max)()
    n = lib.gdn_profile_read(names, 8192, ctypes.cast(ms, ctypes.c_void_p), ctypes.cast(cnt, ctypes.c_void_p), n_max)
    keys = names.value.decode().split("\n")[:n]
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(keys)}


def diag_ut_solve(A):
    """Diagnostic: the chunked path's (I + A)^{-1} for one strictly lower 64 x 64 fp32 matrix."""
    lib = load_library()
    _need_cuda(A)
    T = torch.full((64, 64), float("nan"), dtype=torch.float32, device=A.device)
    _check(lib.gdn_diag_ut_solve(_ptr(A), _ptr(T), _stream()))
    return T
