"""GB300 (sm_103a) fused attention: Python binding of the C ABI in include/gbattn.h.

Only argument marshalling happens here; every step of the computation runs in
the library's CUDA kernels.  torch is used for device memory and streams.  If
the library is missing or cannot be loaded, or an operation reports an error,
an exception is raised -- there is no fallback implementation.

    o, lse = attn_fwd(q, k, v, causal=True)                  # [B,H,T,D] bf16 CUDA tensors
    o, lse = paged_attn_decode(q, k_pool, v_pool, block_table, seq_lens, max_seq_len)

From a projection's rows to those calls, norm and rotation included, and the cache in
4 bits instead of 16:

    q, k, v = qkv_norm_rope(q_rows, k_rows, v_rows, cos_sin, q_weight, k_weight)
    q, new_lens = paged_qkv_append(q_rows, k_rows, v_rows, k_pool, v_pool, block_table,
                                   seq_lens, cos_sin, q_weight, k_weight)
    q, new_lens = paged_kv4_append(q_rows, k_rows, v_rows, kv_pool, block_table, seq_lens,
                                   cos_sin, q_weight, k_weight)
"""

from __future__ import annotations

import ctypes
import math
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgbattn.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_DEVICE = 4

EXPORTS = (
    "attn_status_string",
    "attn_fwd",
    "paged_attn_decode_workspace_size",
    "paged_attn_decode",
    "paged_attn_decode_noalloc",
    "paged_attn_prefill",
    "paged_kv_append",
    "paged_kv_gather",
    "qkv_norm_rope",
    "qkv_norm_rope_bwd_workspace_size",
    "qkv_norm_rope_bwd",
    "paged_qkv_append",
    "paged_kv4_append",
    "paged_kv4_gather",
    "paged_kv4_attn_decode_workspace_size",
    "paged_kv4_attn_decode",
    "paged_kv4_attn_prefill",
    "attn_test_set_failure",
    "attn_device_status",
    "attn_version",
)

_lock = threading.Lock()
_lib = None


class GbAttnError(RuntimeError):
    def __init__(self, op: str, status: int, detail: str = ""):
        self.status = status
        name = status_string(status) if _lib is not None else str(status)
        super().__init__(f"{op} failed: {name}{(' (' + detail + ')') if detail else ''}")


def lib(build_if_missing: bool = True):
    """The loaded ctypes handle of libgbattn.so (built in-tree on first use)."""
    global _lib
    with _lock:
        if _lib is None:
            if build_if_missing:
                from . import build as _build
                _build.build()
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"libgbattn.so not found at {LIB_PATH}; run build.py")
            h = ctypes.CDLL(LIB_PATH)
            _bind(h)
            _lib = h
    return _lib


def _bind(h):
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    h.attn_status_string.argtypes = [I]
    h.attn_status_string.restype = ctypes.c_char_p
    h.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, P]
    h.attn_fwd.restype = I
    h.paged_attn_decode_workspace_size.argtypes = [I, I, I, I]
    h.paged_attn_decode_workspace_size.restype = Z
    h.paged_attn_decode.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, Z, P]
    h.paged_attn_decode.restype = I
    h.paged_attn_decode_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P]
    h.paged_attn_decode_noalloc.restype = I
    h.paged_attn_prefill.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, P, P, P]
    h.paged_attn_prefill.restype = I
    h.paged_kv_append.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
    h.paged_kv_append.restype = I
    h.paged_kv_gather.argtypes = [P, P, P, I, I, I, I, I, I, I, P, P]
    h.paged_kv_gather.restype = I
    S = ctypes.POINTER(ctypes.c_int64)  # three host strides
    h.qkv_norm_rope.argtypes = [P] * 3 + [S] * 3 + [P] * 4 + [I] * 8 + [F] + [P] * 4
    h.qkv_norm_rope.restype = I
    h.qkv_norm_rope_bwd_workspace_size.argtypes = [I, I, I]
    h.qkv_norm_rope_bwd_workspace_size.restype = Z
    h.qkv_norm_rope_bwd.argtypes = ([P] * 5 + [S] * 2 + [P] * 4 + [I] * 8 + [F] + [P] * 3 +
                                    [S] * 3 + [P] * 3 + [Z, P])
    h.qkv_norm_rope_bwd.restype = I
    append = [P] * 3 + [S] * 3 + [P] * 4
    sizes = [P] * 3 + [I] * 11 + [F] + [P] * 2
    h.paged_qkv_append.argtypes = append + [P] * 2 + sizes
    h.paged_qkv_append.restype = I
    h.paged_kv4_append.argtypes = append + [P] + sizes
    h.paged_kv4_append.restype = I
    h.paged_kv4_gather.argtypes = [P, P, P, I, I, I, I, I, I, I, P, P, P]
    h.paged_kv4_gather.restype = I
    h.paged_kv4_attn_decode_workspace_size.argtypes = [I, I, I, I]
    h.paged_kv4_attn_decode_workspace_size.restype = Z
    h.paged_kv4_attn_decode.argtypes = [P] * 4 + [I] * 8 + [F, P, P, P, Z, P]
    h.paged_kv4_attn_decode.restype = I
    h.paged_kv4_attn_prefill.argtypes = [P] * 4 + [I] * 10 + [F, P, P, P]
    h.paged_kv4_attn_prefill.restype = I
    h.attn_test_set_failure.argtypes = [ctypes.c_ulonglong, I]
    h.attn_test_set_failure.restype = I
    h.attn_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    h.attn_device_status.restype = I
    h.attn_version.argtypes = []
    h.attn_version.restype = I


def status_string(status: int) -> str:
    return lib().attn_status_string(int(status)).decode()


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check_tensor(name, t, dtype, shape, device):
    """Metadata checks only (no device access): type, dtype, exact shape, layout, device."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _check_bf16(name, t, ndim, device):
    import torch
    if isinstance(t, torch.Tensor) and t.dim() != ndim:
        raise ValueError(f"{name} must be a {ndim}-d tensor")
    _check_tensor(name, t, torch.bfloat16, None, device)


def _require_cuda(device):
    if device.type != "cuda":
        raise ValueError(f"tensors must be CUDA tensors, got {device}")


def attn_fwd(q, k, v, causal: bool = True, scale: float | None = None, out=None, lse=None,
             return_lse: bool = True, stream=None):
    """Fused attention forward through the C ABI.

    q [B,Hq,T,D], k/v [B,Hkv,T,D] bf16 CUDA tensors -> (o [B,Hq,T,D] bf16,
    lse [B,Hq,T] fp32 or None).  ``scale`` defaults to 1/sqrt(D).  ``out`` and
    ``lse``, when given, must be contiguous tensors of exactly those shapes and
    dtypes on q's device.
    """
    import torch
    device = q.device if isinstance(q, torch.Tensor) else None
    _check_bf16("q", q, 4, device)
    _check_bf16("k", k, 4, device)
    _check_bf16("v", v, 4, device)
    B, Hq, T, D = q.shape
    if k.shape[0] != B or k.shape[2] != T or k.shape[3] != D or v.shape != k.shape:
        raise ValueError("k/v must be [B, Hkv, T, D] matching q")
    Hkv = k.shape[1]
    if out is not None:
        _check_tensor("out", out, torch.bfloat16, (B, Hq, T, D), device)
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, (B, Hq, T), device)
    _require_cuda(device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(device):
        if out is None:
            out = torch.empty_like(q)
        if return_lse and lse is None:
            lse = torch.empty((B, Hq, T), dtype=torch.float32, device=device)
        st = lib().attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            lse.data_ptr() if lse is not None else None, B, Hq, Hkv, T, D,
                            int(bool(causal)), float(scale), _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("attn_fwd", st)
    return out, lse


def paged_attn_decode_workspace_size(num_seqs: int, Hq: int, D: int, max_seq_len: int) -> int:
    return int(lib().paged_attn_decode_workspace_size(num_seqs, Hq, D, max_seq_len))


def paged_attn_decode(q, k_pool, v_pool, block_table, seq_lens, max_seq_len: int,
                      scale: float | None = None, out=None, lse=None, workspace=None,
                      return_lse: bool = True, stream=None):
    """Single-token decode against a paged KV cache through the C ABI.

    q [S,Hq,D] bf16, k_pool/v_pool [NB,Hkv,16,D] bf16, block_table [S,max_blocks]
    int32, seq_lens [S] int32 (all CUDA) -> (o [S,Hq,D] bf16, lse [S,Hq] fp32).
    ``workspace`` (uint8 CUDA tensor) is allocated here when not given.
    """
    import torch
    device = q.device if isinstance(q, torch.Tensor) else None
    _check_bf16("q", q, 3, device)
    _check_bf16("k_pool", k_pool, 4, device)
    _check_bf16("v_pool", v_pool, 4, device)
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    S, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_pool.shape
    if D2 != D or v_pool.shape != k_pool.shape or block_table.dim() != 2 or \
            block_table.shape[0] != S or tuple(seq_lens.shape) != (S,):
        raise ValueError("inconsistent paged-decode shapes")
    if out is not None:
        _check_tensor("out", out, torch.bfloat16, (S, Hq, D), device)
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, (S, Hq), device)
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, None, device)
    _require_cuda(device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    need = paged_attn_decode_workspace_size(S, Hq, D, max_seq_len)
    with torch.cuda.device(device):
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        if out is None:
            out = torch.empty_like(q)
        if return_lse and lse is None:
            lse = torch.empty((S, Hq), dtype=torch.float32, device=device)
        st = lib().paged_attn_decode(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                     block_table.data_ptr(), seq_lens.data_ptr(), bs, S, Hq, Hkv,
                                     D, block_table.shape[1], NB, int(max_seq_len), float(scale),
                                     out.data_ptr(),
                                     lse.data_ptr() if lse is not None else None,
                                     workspace.data_ptr(), workspace.numel(),
                                     _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("paged_attn_decode", st)
    return out, lse


def paged_attn_prefill(q, k_pool, v_pool, block_table, kv_lens, max_kv_len: int,
                       causal: bool = True, scale: float | None = None, out=None, lse=None,
                       return_lse: bool = True, stream=None):
    """Chunked prefill against a paged KV cache through the C ABI.

    q [B,Hq,Tq,D] bf16 (the Tq newest tokens of each item), k_pool/v_pool
    [NB,Hkv,16,D] bf16, block_table [B,max_blocks] int32, kv_lens [B] int32 (all
    CUDA) -> (o [B,Hq,Tq,D] bf16, lse [B,Hq,Tq] fp32).  Query i of item b sits at
    logical position kv_lens[b] - Tq + i.
    """
    import torch
    device = q.device if isinstance(q, torch.Tensor) else None
    _check_bf16("q", q, 4, device)
    _check_bf16("k_pool", k_pool, 4, device)
    _check_bf16("v_pool", v_pool, 4, device)
    for name, t in (("block_table", block_table), ("kv_lens", kv_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    B, Hq, Tq, D = q.shape
    NB, Hkv, bs, D2 = k_pool.shape
    if D2 != D or v_pool.shape != k_pool.shape or block_table.dim() != 2 or \
            block_table.shape[0] != B or tuple(kv_lens.shape) != (B,):
        raise ValueError("inconsistent paged-prefill shapes")
    if out is not None:
        _check_tensor("out", out, torch.bfloat16, (B, Hq, Tq, D), device)
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, (B, Hq, Tq), device)
    _require_cuda(device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(device):
        if out is None:
            out = torch.empty_like(q)
        if return_lse and lse is None:
            lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=device)
        st = lib().paged_attn_prefill(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                      block_table.data_ptr(), kv_lens.data_ptr(), bs, B, Hq, Hkv,
                                      Tq, D, block_table.shape[1], NB, int(max_kv_len),
                                      int(bool(causal)), float(scale), out.data_ptr(),
                                      lse.data_ptr() if lse is not None else None,
                                      _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("paged_attn_prefill", st)
    return out, lse


def paged_kv_append(k_new, v_new, k_pool, v_pool, block_table, seq_lens, new_seq_lens=None,
                    stream=None):
    """Writes the Tn new tokens of each request into the paged pools (in place).

    k_new/v_new [S,Hkv,Tn,D] bf16, k_pool/v_pool [NB,Hkv,16,D] bf16, block_table
    [S,max_blocks] int32, seq_lens [S] int32 (lengths before the append);
    new_seq_lens [S] int32, if given, receives seq_lens + Tn.
    """
    import torch
    device = k_new.device if isinstance(k_new, torch.Tensor) else None
    _check_bf16("k_new", k_new, 4, device)
    _check_bf16("v_new", v_new, 4, device)
    _check_bf16("k_pool", k_pool, 4, device)
    _check_bf16("v_pool", v_pool, 4, device)
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    S, Hkv, Tn, D = k_new.shape
    NB, Hkv2, bs, D2 = k_pool.shape
    if v_new.shape != k_new.shape or v_pool.shape != k_pool.shape or Hkv2 != Hkv or D2 != D or \
            block_table.dim() != 2 or block_table.shape[0] != S or tuple(seq_lens.shape) != (S,):
        raise ValueError("inconsistent append shapes")
    if new_seq_lens is not None:
        _check_tensor("new_seq_lens", new_seq_lens, torch.int32, (S,), device)
    _require_cuda(device)
    with torch.cuda.device(device):
        st = lib().paged_kv_append(k_new.data_ptr(), v_new.data_ptr(), k_pool.data_ptr(),
                                   v_pool.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                                   new_seq_lens.data_ptr() if new_seq_lens is not None else None,
                                   bs, S, Hkv, Tn, D, block_table.shape[1], NB,
                                   _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("paged_kv_append", st)
    return new_seq_lens


def paged_kv_gather(pool, block_table, seq_lens, max_seq_len: int, out=None, stream=None):
    """Each request's cached rows in logical order: out [S,Hkv,max_seq_len,D] bf16
    (rows past a request's length are left as they were)."""
    import torch
    device = pool.device if isinstance(pool, torch.Tensor) else None
    _check_bf16("pool", pool, 4, device)
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    NB, Hkv, bs, D = pool.shape
    S = seq_lens.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("inconsistent gather shapes")
    if out is not None:
        _check_tensor("out", out, torch.bfloat16, (S, Hkv, max_seq_len, D), device)
    _require_cuda(device)
    with torch.cuda.device(device):
        if out is None:
            out = torch.zeros((S, Hkv, max_seq_len, D), dtype=torch.bfloat16, device=device)
        st = lib().paged_kv_gather(pool.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                                   bs, S, Hkv, D, block_table.shape[1], NB, int(max_seq_len),
                                   out.data_ptr(), _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("paged_kv_gather", st)
    return out


def _check_rows(name, t, shape, device):
    """A [B, T, H, D] bf16 operand with any strides but contiguous channels; `shape` may
    hold None for a free dimension.  Metadata checks only."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 4 or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name} must have contiguous channels")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _strides(t):
    """Batch, token and head strides for the C ABI (0 where a dimension has one entry)."""
    if t is None:
        return None
    return (ctypes.c_int64 * 3)(*(st if n > 1 else 0 for n, st in zip(t.shape[:3], t.stride()[:3])))


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _check_rope(cos_sin, q_weight, k_weight, positions, B, T, D, device):
    """Checks the norm and rotation operands; returns (rot_dim, max_pos)."""
    import torch
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check_tensor(name, w, torch.bfloat16, (D,), device)
    if positions is not None:
        _check_tensor("positions", positions, torch.int32, (B, T), device)
    if cos_sin is None:
        return 0, 0
    _check_tensor("cos_sin", cos_sin, torch.float32, None, device)
    if cos_sin.dim() != 2 or cos_sin.shape[0] == 0 or cos_sin.shape[1] == 0:
        raise ValueError("cos_sin must be a non-empty [max_pos, rot_dim] table")
    return cos_sin.shape[1], cos_sin.shape[0]


def _first(*tensors):
    for t in tensors:
        if t is not None:
            return t
    raise ValueError("at least one operand is needed")


def qkv_norm_rope(q, k, v=None, cos_sin=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                  interleaved: bool = False, positions=None, q_out=None, k_out=None, v_out=None,
                  stream=None):
    """RMS norm of every query and key head, rotation, and the move to attn_fwd's layout.

    q [B,T,Hq,D], k/v [B,T,Hkv,D] bf16 CUDA tensors with any batch, token and head
    strides (views of a fused projection) -> (q_out [B,Hq,T,D], k_out, v_out
    [B,Hkv,T,D]).  Each of q, k and v may be None and then comes back as None.
    ``cos_sin`` [max_pos, rot_dim] fp32 holds rot_dim / 2 cosines, then the sines, of
    each position (None: no rotation); ``q_weight``/``k_weight`` [D] bf16 (None: no
    norm); ``positions`` [B,T] int32 (None: 0 .. T-1).
    """
    import torch
    some = _first(q, k, v)
    device = some.device if isinstance(some, torch.Tensor) else None
    kv = k if k is not None else v
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is not None:
            _check_rows(name, t, (None,) * 4, device)
    B, T, _, D = some.shape
    for name, t, heads in (("q", q, None), ("k", k, None), ("v", v, None if kv is v else kv.shape[2])):
        if t is not None:
            _check_rows(name, t, (B, T, heads, D), device)
    rot, max_pos = _check_rope(cos_sin, q_weight, k_weight, positions, B, T, D, device)
    for name, t, src in (("q_out", q_out, q), ("k_out", k_out, k), ("v_out", v_out, v)):
        if t is not None:
            if src is None:
                raise ValueError(f"{name} is given without its input")
            _check_tensor(name, t, torch.bfloat16, (B, src.shape[2], T, D), device)
    _require_cuda(device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        def out(t, src):
            if t is not None or src is None:
                return t
            return torch.empty((B, src.shape[2], T, D), dtype=torch.bfloat16, device=device)
        q_out, k_out, v_out = out(q_out, q), out(k_out, k), out(v_out, v)
        st = lib().qkv_norm_rope(_ptr(q), _ptr(k), _ptr(v), _strides(q), _strides(k), _strides(v),
                                 _ptr(q_weight), _ptr(k_weight), _ptr(cos_sin), _ptr(positions),
                                 B, T, q.shape[2] if q is not None else 0,
                                 kv.shape[2] if kv is not None else 0, D, rot, max_pos,
                                 int(bool(interleaved)), float(eps), _ptr(q_out), _ptr(k_out),
                                 _ptr(v_out), _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("qkv_norm_rope", st)
    return q_out, k_out, v_out


def qkv_norm_rope_bwd_workspace_size(B: int, T: int, D: int) -> int:
    return int(lib().qkv_norm_rope_bwd_workspace_size(B, T, D))


def qkv_norm_rope_bwd(dq_out, dk_out, dv_out=None, q=None, k=None, cos_sin=None, q_weight=None,
                      k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                      positions=None, dq=None, dk=None, dv=None, dq_weight=None, dk_weight=None,
                      workspace=None, stream=None):
    """Gradients of qkv_norm_rope: (dq, dk, dv, dq_weight, dk_weight).

    dq_out [B,Hq,T,D], dk_out/dv_out [B,Hkv,T,D] bf16; q and k are the forward's inputs
    (needed with a weight).  dq, dk, dv are [B,T,H,D] bf16 and may be strided views
    without overlap; when none is given they are views of one [B,T,all heads,D] buffer,
    the gradient of a fused projection.  The weight gradients [D] are fp32, None for an
    operand without a weight.
    """
    import torch
    some = _first(dq_out, dk_out, dv_out)
    device = some.device if isinstance(some, torch.Tensor) else None
    for name, t in (("dq_out", dq_out), ("dk_out", dk_out), ("dv_out", dv_out)):
        if t is not None:
            _check_bf16(name, t, 4, device)
    B, _, T, D = some.shape
    kv = dk_out if dk_out is not None else dv_out
    Hq = dq_out.shape[1] if dq_out is not None else 0
    Hkv = kv.shape[1] if kv is not None else 0
    for name, t, heads in (("dq_out", dq_out, Hq), ("dk_out", dk_out, Hkv), ("dv_out", dv_out, Hkv)):
        if t is not None and tuple(t.shape) != (B, heads, T, D):
            raise ValueError(f"{name} must have shape {(B, heads, T, D)}, got {tuple(t.shape)}")
    rot, max_pos = _check_rope(cos_sin, q_weight, k_weight, positions, B, T, D, device)
    for name, x, w, heads in (("q", q, q_weight, Hq), ("k", k, k_weight, Hkv)):
        if w is None:
            continue
        if x is None:
            raise ValueError(f"{name} is needed for the gradient of its norm")
        _check_rows(name, x, (B, T, heads, D), device)
    for name, t, heads, g in (("dq", dq, Hq, dq_out), ("dk", dk, Hkv, dk_out),
                              ("dv", dv, Hkv, dv_out)):
        if t is not None:
            if g is None:
                raise ValueError(f"{name} is given without the gradient of its output")
            _check_rows(name, t, (B, T, heads, D), device)
    for name, t, w in (("dq_weight", dq_weight, q_weight), ("dk_weight", dk_weight, k_weight)):
        if t is not None:
            if w is None:
                raise ValueError(f"{name} is given without its weight")
            _check_tensor(name, t, torch.float32, (D,), device)
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, None, device)
    _require_cuda(device)
    if q_weight is None:
        q = None
    if k_weight is None:
        k = None
    with torch.cuda.device(device), torch.cuda.stream(stream):
        if dq is None and dk is None and dv is None:
            sizes = [Hq if dq_out is not None else 0, Hkv if dk_out is not None else 0,
                     Hkv if dv_out is not None else 0]
            fused = torch.empty((B, T, sum(sizes), D), dtype=torch.bfloat16, device=device)
            dq, dk, dv = (t if n else None for t, n in zip(fused.split(sizes, 2), sizes))

        def rows(t, g):
            if t is not None or g is None:
                return t
            return torch.empty((B, T, g.shape[1], D), dtype=torch.bfloat16, device=device)

        def vector(t, w):
            if t is not None or w is None:
                return t
            return torch.empty((D,), dtype=torch.float32, device=device)
        dq, dk, dv = rows(dq, dq_out), rows(dk, dk_out), rows(dv, dv_out)
        dq_weight, dk_weight = vector(dq_weight, q_weight), vector(dk_weight, k_weight)
        if workspace is None and (q_weight is not None or k_weight is not None):
            need = qkv_norm_rope_bwd_workspace_size(B, T, D)
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        st = lib().qkv_norm_rope_bwd(_ptr(dq_out), _ptr(dk_out), _ptr(dv_out), _ptr(q), _ptr(k),
                                     _strides(q), _strides(k), _ptr(q_weight), _ptr(k_weight),
                                     _ptr(cos_sin), _ptr(positions), B, T, Hq, Hkv, D, rot,
                                     max_pos, int(bool(interleaved)), float(eps), _ptr(dq),
                                     _ptr(dk), _ptr(dv), _strides(dq), _strides(dk), _strides(dv),
                                     _ptr(dq_weight), _ptr(dk_weight), _ptr(workspace),
                                     workspace.numel() if workspace is not None else 0,
                                     _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("qkv_norm_rope_bwd", st)
    return dq, dk, dv, dq_weight, dk_weight


def _append(op, pools, q, k, v, block_table, seq_lens, cos_sin, q_weight, k_weight, eps,
            interleaved, positions, q_out, new_seq_lens, stream):
    import torch
    device = k.device if isinstance(k, torch.Tensor) else None
    _check_rows("k", k, (None,) * 4, device)
    S, Tn, Hkv, D = k.shape
    _check_rows("v", v, (S, Tn, Hkv, D), device)
    if q is not None:
        _check_rows("q", q, (S, Tn, None, D), device)
    Hq = q.shape[2] if q is not None else 0
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    if block_table.dim() != 2 or block_table.shape[0] != S or tuple(seq_lens.shape) != (S,):
        raise ValueError("inconsistent append shapes")
    if len(pools) == 2:
        for name, t in zip(("k_pool", "v_pool"), pools):
            _check_bf16(name, t, 4, device)
        NB, Hkv2, bs, D2 = pools[0].shape
        if pools[1].shape != pools[0].shape or Hkv2 != Hkv or D2 != D:
            raise ValueError("inconsistent append shapes")
    else:
        NB, bs = _check_kv4("kv_pool", pools[0], Hkv, D, device), 16
    rot, max_pos = _check_rope(cos_sin, q_weight, k_weight, positions, S, Tn, D, device)
    if q_out is not None:
        if q is None:
            raise ValueError("q_out is given without q")
        _check_tensor("q_out", q_out, torch.bfloat16, (S, Hq, Tn, D), device)
    if new_seq_lens is not None:
        _check_tensor("new_seq_lens", new_seq_lens, torch.int32, (S,), device)
    _require_cuda(device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        if q is not None and q_out is None:
            q_out = torch.empty((S, Hq, Tn, D), dtype=torch.bfloat16, device=device)
        st = getattr(lib(), op)(_ptr(q), _ptr(k), _ptr(v), _strides(q), _strides(k), _strides(v),
                                _ptr(q_weight), _ptr(k_weight), _ptr(cos_sin), _ptr(positions),
                                *(_ptr(t) for t in pools), block_table.data_ptr(),
                                seq_lens.data_ptr(), _ptr(new_seq_lens), bs, S, Tn, Hq, Hkv, D,
                                block_table.shape[1], NB, rot, max_pos, int(bool(interleaved)),
                                float(eps), _ptr(q_out), _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError(op, st)
    return q_out, new_seq_lens


def paged_qkv_append(q, k, v, k_pool, v_pool, block_table, seq_lens, cos_sin=None, q_weight=None,
                     k_weight=None, eps: float = 1e-6, interleaved: bool = False, positions=None,
                     q_out=None, new_seq_lens=None, stream=None):
    """Norm, rotation and append of each request's Tn new tokens in one pass.

    q [S,Tn,Hq,D] (None: no queries), k/v [S,Tn,Hkv,D] bf16 with any strides as in
    qkv_norm_rope; k_pool/v_pool [NB,Hkv,16,D] bf16 are written in place.  Token t of
    request r is rotated by its place in the cache, seq_lens[r] + t, unless
    ``positions`` [S,Tn] int32 says otherwise.  Returns (q_out [S,Hq,Tn,D] or None,
    new_seq_lens); new_seq_lens [S] int32, if given, receives seq_lens + Tn.
    """
    return _append("paged_qkv_append", (k_pool, v_pool), q, k, v, block_table, seq_lens, cos_sin,
                   q_weight, k_weight, eps, interleaved, positions, q_out, new_seq_lens, stream)


def _check_kv4(name, pool, Hkv, D, device):
    """A 4-bit pool [NB, Hkv, 18 D] uint8; returns NB."""
    import torch
    if isinstance(pool, torch.Tensor) and pool.dim() != 3:
        raise ValueError(f"{name} must be a 3-d tensor")
    _check_tensor(name, pool, torch.uint8, None, device)
    if Hkv is not None and (pool.shape[1] != Hkv or pool.shape[2] != 18 * D):
        raise ValueError(f"{name} must have shape (blocks, {Hkv}, {18 * D}), got {tuple(pool.shape)}")
    if pool.shape[2] % 18 != 0:
        raise ValueError(f"{name} must have 18 D bytes per block and head, got {pool.shape[2]}")
    return pool.shape[0]


def paged_kv4_append(q, k, v, kv_pool, block_table, seq_lens, cos_sin=None, q_weight=None,
                     k_weight=None, eps: float = 1e-6, interleaved: bool = False, positions=None,
                     q_out=None, new_seq_lens=None, stream=None):
    """paged_qkv_append into the 4-bit cache: kv_pool [NB,Hkv,18*D] uint8 is written in
    place (the format is described in include/gbattn.h)."""
    return _append("paged_kv4_append", (kv_pool,), q, k, v, block_table, seq_lens, cos_sin,
                   q_weight, k_weight, eps, interleaved, positions, q_out, new_seq_lens, stream)


def paged_kv4_gather(kv_pool, block_table, seq_lens, max_seq_len: int, k_out=None, v_out=None,
                     stream=None):
    """The values the 4-bit cache holds, in logical order: k_out, v_out
    [S,Hkv,max_seq_len,D] bf16 (rows past a request's length are left as they were)."""
    import torch
    device = kv_pool.device if isinstance(kv_pool, torch.Tensor) else None
    NB = _check_kv4("kv_pool", kv_pool, None, None, device)
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    Hkv, D = kv_pool.shape[1], kv_pool.shape[2] // 18
    S = seq_lens.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] != S or seq_lens.dim() != 1:
        raise ValueError("inconsistent gather shapes")
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _check_tensor(name, t, torch.bfloat16, (S, Hkv, max_seq_len, D), device)
    _require_cuda(device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        def out(t):
            if t is not None:
                return t
            return torch.zeros((S, Hkv, max_seq_len, D), dtype=torch.bfloat16, device=device)
        k_out, v_out = out(k_out), out(v_out)
        st = lib().paged_kv4_gather(kv_pool.data_ptr(), block_table.data_ptr(),
                                    seq_lens.data_ptr(), 16, S, Hkv, D, block_table.shape[1], NB,
                                    int(max_seq_len), k_out.data_ptr(), v_out.data_ptr(),
                                    _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("paged_kv4_gather", st)
    return k_out, v_out


def paged_kv4_attn_decode_workspace_size(num_seqs: int, Hq: int, D: int, max_seq_len: int) -> int:
    return int(lib().paged_kv4_attn_decode_workspace_size(num_seqs, Hq, D, max_seq_len))


def paged_kv4_attn_decode(q, kv_pool, block_table, seq_lens, max_seq_len: int,
                          scale: float | None = None, out=None, lse=None, workspace=None,
                          return_lse: bool = True, stream=None):
    """Single-token decode against the 4-bit paged cache through the C ABI.

    q [S,Hq,D] bf16, kv_pool [NB,Hkv,18*D] uint8, block_table [S,max_blocks] int32,
    seq_lens [S] int32 (all CUDA) -> (o [S,Hq,D] bf16, lse [S,Hq] fp32).
    ``workspace`` (uint8 CUDA tensor) is allocated here when not given.
    """
    import torch
    device = q.device if isinstance(q, torch.Tensor) else None
    _check_bf16("q", q, 3, device)
    S, Hq, D = q.shape
    NB = _check_kv4("kv_pool", kv_pool, None, None, device)
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    if kv_pool.shape[2] != 18 * D or block_table.dim() != 2 or block_table.shape[0] != S or \
            tuple(seq_lens.shape) != (S,):
        raise ValueError("inconsistent paged-decode shapes")
    if out is not None:
        _check_tensor("out", out, torch.bfloat16, (S, Hq, D), device)
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, (S, Hq), device)
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, None, device)
    _require_cuda(device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        if workspace is None:
            need = paged_kv4_attn_decode_workspace_size(S, Hq, D, max_seq_len)
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        if out is None:
            out = torch.empty_like(q)
        if return_lse and lse is None:
            lse = torch.empty((S, Hq), dtype=torch.float32, device=device)
        st = lib().paged_kv4_attn_decode(q.data_ptr(), kv_pool.data_ptr(), block_table.data_ptr(),
                                         seq_lens.data_ptr(), 16, S, Hq, kv_pool.shape[1], D,
                                         block_table.shape[1], NB, int(max_seq_len), float(scale),
                                         out.data_ptr(), _ptr(lse), workspace.data_ptr(),
                                         workspace.numel(), _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("paged_kv4_attn_decode", st)
    return out, lse


def paged_kv4_attn_prefill(q, kv_pool, block_table, kv_lens, max_kv_len: int,
                           causal: bool = True, scale: float | None = None, out=None, lse=None,
                           return_lse: bool = True, stream=None):
    """Chunked prefill against the 4-bit paged cache through the C ABI.

    q [B,Hq,Tq,D] bf16 (the Tq newest tokens of each item), kv_pool [NB,Hkv,18*D]
    uint8, block_table [B,max_blocks] int32, kv_lens [B] int32 (all CUDA) -> (o
    [B,Hq,Tq,D] bf16, lse [B,Hq,Tq] fp32).  Query i of item b sits at logical
    position kv_lens[b] - Tq + i.
    """
    import torch
    device = q.device if isinstance(q, torch.Tensor) else None
    _check_bf16("q", q, 4, device)
    B, Hq, Tq, D = q.shape
    NB = _check_kv4("kv_pool", kv_pool, None, None, device)
    for name, t in (("block_table", block_table), ("kv_lens", kv_lens)):
        _check_tensor(name, t, torch.int32, None, device)
    if kv_pool.shape[2] != 18 * D or block_table.dim() != 2 or block_table.shape[0] != B or \
            tuple(kv_lens.shape) != (B,):
        raise ValueError("inconsistent paged-prefill shapes")
    if out is not None:
        _check_tensor("out", out, torch.bfloat16, (B, Hq, Tq, D), device)
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, (B, Hq, Tq), device)
    _require_cuda(device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        if out is None:
            out = torch.empty_like(q)
        if return_lse and lse is None:
            lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=device)
        st = lib().paged_kv4_attn_prefill(q.data_ptr(), kv_pool.data_ptr(),
                                          block_table.data_ptr(), kv_lens.data_ptr(), 16, B, Hq,
                                          kv_pool.shape[1], Tq, D, block_table.shape[1], NB,
                                          int(max_kv_len), int(bool(causal)), float(scale),
                                          out.data_ptr(), _ptr(lse),
                                          _stream_handle(stream, device))
    if st != ATTN_OK:
        raise GbAttnError("paged_kv4_attn_prefill", st)
    return out, lse


def test_set_failure(wait_limit_ns: int = 0, withhold_copy: bool = False) -> None:
    """Test hook: in-kernel wait limit (0 = default 2 s) and whether the next kernels'
    copy warps withhold their first copy so that a wait runs out."""
    st = lib().attn_test_set_failure(int(wait_limit_ns), int(bool(withhold_copy)))
    if st != ATTN_OK:
        raise GbAttnError("attn_test_set_failure", st)


def attn_device_status():
    """(status, flags): synchronises the current device, reads and clears its flag word."""
    flags = ctypes.c_uint(0)
    st = lib().attn_device_status(ctypes.byref(flags))
    return st, flags.value


def version() -> str:
    v = lib().attn_version()
    return f"{v // 10000}.{(v // 100) % 100}.{v % 100}"
