"""GB300 (sm_103a) fused attention: Python binding of the C ABI in include/gbattn.h.

Only argument marshalling happens here (for the usual call of the newer operators in
_binding, compiled from csrc/binding.cpp); every step of the computation runs in
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
import functools
import importlib
import math
import os
import threading
import warnings

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
    "paged_kv4_attn_prefill_workspace_size",
    "paged_kv4_attn_prefill",
    "attn_test_set_failure",
    "attn_device_status",
    "attn_version",
)

_lock = threading.Lock()
_lib = None
_torch = _Tensor = _bf16 = _f32 = _i32 = _u8 = _quick = None  # set by _load_torch


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
    h.paged_kv4_attn_decode_workspace_size.argtypes = [I, I, I, I, I]
    h.paged_kv4_attn_decode_workspace_size.restype = Z
    h.paged_kv4_attn_decode.argtypes = [P] * 4 + [I] * 8 + [F, P, P, P, Z, P]
    h.paged_kv4_attn_decode.restype = I
    h.paged_kv4_attn_prefill_workspace_size.argtypes = [I, I, I, I, I, I]
    h.paged_kv4_attn_prefill_workspace_size.restype = Z
    h.paged_kv4_attn_prefill.argtypes = [P] * 4 + [I] * 10 + [F, P, P, P, Z, P]
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


# The operators below are called between kernels of a few microseconds.  The usual call
# therefore goes through _binding (csrc/binding.cpp), which makes the same checks in compiled
# code and returns None for everything else: other streams and devices, and whatever is
# wrong with the arguments, which the Python code then handles and names.  (Host time of a
# paged_qkv_append, whose kernel runs for 3 us: 5.2 us, and 25 us the long way.)

class _On:
    """The device, and the stream if one is given, current for allocations and launches
    (outputs and workspaces then belong to that stream's memory pool)."""

    __slots__ = ("device", "stream", "inner")

    def __init__(self, device, stream):
        self.device, self.stream, self.inner = device, stream, None

    def __enter__(self):
        if self.stream is not None and self.stream.device != self.device:
            raise ValueError(f"stream must be on {self.device}, got {self.stream.device}")
        if self.stream is not None or _torch.cuda.current_device() != self.device.index:
            self.inner = (_torch.cuda.device(self.device), _torch.cuda.stream(self.stream))
            for c in self.inner:
                c.__enter__()
        if self.stream is not None:
            return self.stream.cuda_stream
        return _torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *exc):
        if self.inner is not None:
            for c in reversed(self.inner):
                c.__exit__(*exc)
        return False


def _check(name, t, dtype, shape, device):
    """_check_tensor, quick where all is well."""
    if t.__class__ is _Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous() and \
            t.device == device:
        return
    _check_tensor(name, t, dtype, shape, device)


def _is_rows(t, device):
    """Whether t is a [B, T, H, D] bf16 operand: any strides but contiguous channels."""
    return (t.__class__ is _Tensor and t.dtype is _bf16 and t.dim() == 4 and
            (t.stride(3) == 1 or t.shape[3] == 1) and t.device == device)


def _check_rows(name, t, shape, device):
    """Raises for what is wrong with a [B, T, H, D] operand; `shape` may hold None for a
    free dimension.  Metadata checks only."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != _bf16:
        raise ValueError(f"{name} must be {_bf16}, got {t.dtype}")
    if t.dim() != 4 or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name} must have contiguous channels")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


@functools.lru_cache(maxsize=1024)
def _stride_array(shape, strides):
    """Batch, token and head strides for the C ABI (0 where a dimension has one entry)."""
    return (ctypes.c_int64 * 3)(*(st if n > 1 else 0 for n, st in zip(shape[:3], strides)))


def _strides(t):
    return _stride_array(t.shape, t.stride()) if t is not None else None


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _check_table(block_table, S, device):
    """A block table [S, blocks]; its width is an int of the C ABI."""
    _check_tensor("block_table", block_table, _i32, None, device)
    if block_table.dim() != 2 or block_table.shape[0] != S or block_table.shape[1] >= 1 << 31:
        raise ValueError(f"block_table must have shape ({S}, blocks), got {tuple(block_table.shape)}")


def _check_rope(cos_sin, q_weight, k_weight, positions, B, T, D, device):
    """Checks the norm and rotation operands; returns (rot_dim, max_pos)."""
    if q_weight is not None:
        _check("q_weight", q_weight, _bf16, (D,), device)
    if k_weight is not None:
        _check("k_weight", k_weight, _bf16, (D,), device)
    if positions is not None:
        _check("positions", positions, _i32, (B, T), device)
    if cos_sin is None:
        return 0, 0
    shape = cos_sin.shape if isinstance(cos_sin, _Tensor) else None
    _check("cos_sin", cos_sin, _f32, shape, device)
    if len(shape) != 2 or shape[0] == 0 or shape[1] == 0 or max(shape) >= 1 << 31:
        raise ValueError("cos_sin must be a non-empty [max_pos, rot_dim] table of sizes below 2^31")
    return shape[1], shape[0]


def _check_no_gradients(op, **operands):
    """Raises for an operand through which torch expects a derivative: outputs carry none."""
    grad_mode, fwd = _torch.is_grad_enabled(), _torch.autograd.forward_ad
    for name, t in operands.items():
        if t is None:
            continue
        if (grad_mode and t.requires_grad) or fwd.unpack_dual(t).tangent is not None:
            raise ValueError(
                f"{op} records nothing for automatic differentiation, and {name} takes part in it: "
                "call it under torch.no_grad() (or in an autograd.Function) and take the "
                "gradients from qkv_norm_rope_bwd")


def _load_torch():
    global _torch, _Tensor, _bf16, _f32, _i32, _u8
    import torch
    _Tensor = torch.Tensor
    _bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    _load_quick(torch)
    _torch = torch  # last: another thread that finds it set finds the rest too


def _load_quick(torch):
    """Binds _quick, the module _binding, to the library and torch's current device
    and stream, if it was built."""
    global _quick
    h = lib()
    if not hasattr(torch._C, "_cuda_getDevice"):  # a torch without CUDA
        return
    try:
        m = importlib.import_module("._binding", __name__)
        names = ("qkv_norm_rope", "qkv_norm_rope_bwd", "qkv_norm_rope_bwd_workspace_size",
                 "paged_qkv_append", "paged_kv4_append", "paged_kv4_gather",
                 "paged_kv4_attn_decode", "paged_kv4_attn_decode_workspace_size",
                 "paged_kv4_attn_prefill", "paged_kv4_attn_prefill_workspace_size")
        m.setup(torch.__version__, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream,
                *(ctypes.cast(getattr(h, n), ctypes.c_void_p).value for n in names))
    except ImportError as e:  # not built, or against another torch
        warnings.warn(f"_binding cannot be used ({e}): calls go through the interpreter, at about "
                      "20 us more of host time each", RuntimeWarning)
        return
    _quick = m


def _done(op, r):
    """The result of a quick call that was made."""
    if r.__class__ is tuple:
        return r
    raise GbAttnError(op, r)


def _first(*tensors):
    """The first operand given, after making sure that it is a tensor."""
    if _torch is None:
        _load_torch()
    for t in tensors:
        if t is not None:
            if not isinstance(t, _Tensor):
                raise TypeError(f"operands must be torch.Tensor, got {type(t)}")
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

    Nothing is recorded for automatic differentiation: qkv_norm_rope_bwd computes the
    gradients.  Where gradients are enabled, operands that require one (and the duals of
    forward mode) are refused; call it under torch.no_grad() or in an autograd.Function.
    """
    if _torch is None:
        _load_torch()
    if _quick is not None and stream is None:
        r = _quick.rope(q, k, v, cos_sin, q_weight, k_weight, eps, interleaved, positions, q_out,
                        k_out, v_out)
        if r is not None:
            return _done("qkv_norm_rope", r)
    some = _first(q, k, v)
    device = some.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is not None and not _is_rows(t, device):
            _check_rows(name, t, (None,) * 4, device)
    B, T, _, D = some.shape
    Hq = q.shape[2] if q is not None else 0
    kv = k if k is not None else v
    Hkv = kv.shape[2] if kv is not None else 0
    for name, t, heads, out in (("q", q, Hq, q_out), ("k", k, Hkv, k_out), ("v", v, Hkv, v_out)):
        if t is None:
            if out is not None:
                raise ValueError(f"{name}_out is given without its input")
            continue
        if t.shape != (B, T, heads, D):
            _check_rows(name, t, (B, T, heads, D), device)
        if out is not None:
            _check(name + "_out", out, _bf16, (B, heads, T, D), device)
    rot, max_pos = _check_rope(cos_sin, q_weight, k_weight, positions, B, T, D, device)
    _check_no_gradients("qkv_norm_rope", q=q, k=k, v=v, cos_sin=cos_sin, q_weight=q_weight,
                        k_weight=k_weight)
    _require_cuda(device)
    with _On(device, stream) as handle:
        if q_out is None and q is not None:
            q_out = _torch.empty((B, Hq, T, D), dtype=_bf16, device=device)
        if k_out is None and k is not None:
            k_out = _torch.empty((B, Hkv, T, D), dtype=_bf16, device=device)
        if v_out is None and v is not None:
            v_out = _torch.empty((B, Hkv, T, D), dtype=_bf16, device=device)
        st = (_lib or lib()).qkv_norm_rope(
            _ptr(q), _ptr(k), _ptr(v), _strides(q), _strides(k), _strides(v), _ptr(q_weight),
            _ptr(k_weight), _ptr(cos_sin), _ptr(positions), B, T, Hq, Hkv, D, rot, max_pos,
            1 if interleaved else 0, float(eps), _ptr(q_out), _ptr(k_out), _ptr(v_out), handle)
    if st != ATTN_OK:
        raise GbAttnError("qkv_norm_rope", st)
    return q_out, k_out, v_out


def qkv_norm_rope_bwd_workspace_size(B: int, T: int, D: int) -> int:
    return (_lib or lib()).qkv_norm_rope_bwd_workspace_size(B, T, D)


def qkv_norm_rope_bwd(dq_out, dk_out, dv_out=None, q=None, k=None, cos_sin=None, q_weight=None,
                      k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                      positions=None, dq=None, dk=None, dv=None, dq_weight=None, dk_weight=None,
                      workspace=None, stream=None):
    """Gradients of qkv_norm_rope: (dq, dk, dv, dq_weight, dk_weight).

    dq_out [B,Hq,T,D], dk_out/dv_out [B,Hkv,T,D] bf16; q and k are the forward's inputs
    (needed with a weight).  dq, dk, dv are [B,T,H,D] bf16 and may be strided views
    without overlap; when none is given they are views of one [B,T,all heads,D] buffer,
    the gradient of a fused projection.  The weight gradients [D] are fp32, None for an
    operand without a weight.  Operands that take part in automatic differentiation are
    refused as in qkv_norm_rope.
    """
    if _torch is None:
        _load_torch()
    if _quick is not None and stream is None and dq is None and dk is None and \
            dv is None and dq_weight is None and dk_weight is None and workspace is None:
        r = _quick.rope_bwd(dq_out, dk_out, dv_out, q, k, cos_sin, q_weight, k_weight, eps,
                            interleaved, positions)
        if r is not None:
            return _done("qkv_norm_rope_bwd", r)
    some = _first(dq_out, dk_out, dv_out)
    device = some.device
    if some.dim() != 4:
        raise ValueError("gradients must be 4-d tensors")
    B, _, T, D = some.shape
    Hq = dq_out.shape[1] if dq_out is not None else 0
    kv = dk_out if dk_out is not None else dv_out
    Hkv = kv.shape[1] if kv is not None and kv.dim() > 1 else 0
    for name, g, d, heads in (("dq", dq_out, dq, Hq), ("dk", dk_out, dk, Hkv),
                              ("dv", dv_out, dv, Hkv)):
        if g is None:
            if d is not None:
                raise ValueError(f"{name} is given without the gradient of its output")
            continue
        _check(name + "_out", g, _bf16, (B, heads, T, D), device)
        if d is not None:
            _check_rows(name, d, (B, T, heads, D), device)
    rot, max_pos = _check_rope(cos_sin, q_weight, k_weight, positions, B, T, D, device)
    for name, x, w, dw, heads in (("q", q, q_weight, dq_weight, Hq),
                                  ("k", k, k_weight, dk_weight, Hkv)):
        if w is None:
            if dw is not None:
                raise ValueError(f"d{name}_weight is given without its weight")
            continue
        if x is None:
            raise ValueError(f"{name} is needed for the gradient of its norm")
        if not _is_rows(x, device) or x.shape != (B, T, heads, D):
            _check_rows(name, x, (B, T, heads, D), device)
        if dw is not None:
            _check(f"d{name}_weight", dw, _f32, (D,), device)
    if workspace is not None:
        _check_tensor("workspace", workspace, _u8, None, device)
    if q_weight is None:
        q = None
    if k_weight is None:
        k = None
    _check_no_gradients("qkv_norm_rope_bwd", dq_out=dq_out, dk_out=dk_out, dv_out=dv_out, q=q, k=k,
                        cos_sin=cos_sin, q_weight=q_weight, k_weight=k_weight)
    _require_cuda(device)
    with _On(device, stream) as handle:
        if dq is None and dk is None and dv is None:
            nq, nk = (Hq if dq_out is not None else 0), (Hkv if dk_out is not None else 0)
            nv = Hkv if dv_out is not None else 0
            fused = _torch.empty((B, T, nq + nk + nv, D), dtype=_bf16, device=device)
            dq = fused[:, :, :nq] if nq else None
            dk = fused[:, :, nq:nq + nk] if nk else None
            dv = fused[:, :, nq + nk:] if nv else None
        else:
            dq, dk, dv = (d if d is not None or g is None else
                          _torch.empty((B, T, g.shape[1], D), dtype=_bf16, device=device)
                          for d, g in ((dq, dq_out), (dk, dk_out), (dv, dv_out)))
        if dq_weight is None and q_weight is not None:
            dq_weight = _torch.empty((D,), dtype=_f32, device=device)
        if dk_weight is None and k_weight is not None:
            dk_weight = _torch.empty((D,), dtype=_f32, device=device)
        if workspace is None and (q_weight is not None or k_weight is not None):
            need = qkv_norm_rope_bwd_workspace_size(B, T, D)
            workspace = _torch.empty((max(need, 256),), dtype=_u8, device=device)
        st = (_lib or lib()).qkv_norm_rope_bwd(
            _ptr(dq_out), _ptr(dk_out), _ptr(dv_out), _ptr(q), _ptr(k), _strides(q), _strides(k),
            _ptr(q_weight), _ptr(k_weight), _ptr(cos_sin), _ptr(positions), B, T, Hq, Hkv, D, rot,
            max_pos, 1 if interleaved else 0, float(eps), _ptr(dq), _ptr(dk), _ptr(dv), _strides(dq),
            _strides(dk), _strides(dv), _ptr(dq_weight), _ptr(dk_weight), _ptr(workspace),
            workspace.numel() if workspace is not None else 0, handle)
    if st != ATTN_OK:
        raise GbAttnError("qkv_norm_rope_bwd", st)
    return dq, dk, dv, dq_weight, dk_weight


def _append(op, pools, q, k, v, block_table, seq_lens, cos_sin, q_weight, k_weight, eps,
            interleaved, positions, q_out, new_seq_lens, stream):
    if _torch is None:
        _load_torch()
    if _quick is not None and stream is None:
        quick = _quick.append4 if op == "paged_kv4_append" else _quick.append
        r = quick(q, k, v, pools[0], pools[1], block_table, seq_lens, cos_sin, q_weight, k_weight,
                  eps, interleaved, positions, q_out, new_seq_lens)
        if r is not None:
            return _done(op, r)
    if op == "paged_kv4_append":
        pools = pools[:1]
    _first(k)
    device = k.device
    if not _is_rows(k, device):
        _check_rows("k", k, (None,) * 4, device)
    S, Tn, Hkv, D = k.shape
    if not _is_rows(v, device) or v.shape != (S, Tn, Hkv, D):
        _check_rows("v", v, (S, Tn, Hkv, D), device)
    Hq = 0
    if q is not None:
        if not _is_rows(q, device):
            _check_rows("q", q, (S, Tn, None, D), device)
        Hq = q.shape[2]
        if q.shape != (S, Tn, Hq, D):
            _check_rows("q", q, (S, Tn, None, D), device)
    _check("seq_lens", seq_lens, _i32, (S,), device)
    _check_table(block_table, S, device)
    if len(pools) == 2:
        _check_bf16("k_pool", pools[0], 4, device)
        shape = pools[0].shape
        _check("v_pool", pools[1], _bf16, shape, device)
        NB, Hkv2, bs, D2 = shape
        if Hkv2 != Hkv or D2 != D:
            raise ValueError("inconsistent append shapes")
    else:
        NB, bs = _check_kv4("kv_pool", pools[0], Hkv, D, device), 16
    rot, max_pos = _check_rope(cos_sin, q_weight, k_weight, positions, S, Tn, D, device)
    if q_out is not None:
        if q is None:
            raise ValueError("q_out is given without q")
        _check("q_out", q_out, _bf16, (S, Hq, Tn, D), device)
    if new_seq_lens is not None:
        _check("new_seq_lens", new_seq_lens, _i32, (S,), device)
    _require_cuda(device)
    with _On(device, stream) as handle:
        if q is not None and q_out is None:
            q_out = _torch.empty((S, Hq, Tn, D), dtype=_bf16, device=device)
        st = getattr(_lib or lib(), op)(
            _ptr(q), k.data_ptr(), v.data_ptr(), _strides(q), _strides(k), _strides(v),
            _ptr(q_weight), _ptr(k_weight), _ptr(cos_sin), _ptr(positions),
            *[t.data_ptr() for t in pools], block_table.data_ptr(), seq_lens.data_ptr(),
            _ptr(new_seq_lens), bs, S, Tn, Hq, Hkv, D, block_table.shape[1], NB, rot, max_pos,
            1 if interleaved else 0, float(eps), _ptr(q_out), handle)
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
    if isinstance(pool, _Tensor) and pool.dim() != 3:
        raise ValueError(f"{name} must be a 3-d tensor")
    _check_tensor(name, pool, _u8, None, device)
    NB, heads, chunk = pool.shape
    if Hkv is not None and (heads != Hkv or chunk != 18 * D):
        raise ValueError(f"{name} must have shape (blocks, {Hkv}, {18 * D}), got {tuple(pool.shape)}")
    if chunk % 18 != 0:
        raise ValueError(f"{name} must have 18 D bytes per block and head, got {chunk}")
    return NB


def paged_kv4_append(q, k, v, kv_pool, block_table, seq_lens, cos_sin=None, q_weight=None,
                     k_weight=None, eps: float = 1e-6, interleaved: bool = False, positions=None,
                     q_out=None, new_seq_lens=None, stream=None):
    """paged_qkv_append into the 4-bit cache: kv_pool [NB,Hkv,18*D] uint8 is written in
    place (the format is described in include/gbattn.h)."""
    return _append("paged_kv4_append", (kv_pool, None), q, k, v, block_table, seq_lens, cos_sin,
                   q_weight, k_weight, eps, interleaved, positions, q_out, new_seq_lens, stream)


def paged_kv4_gather(kv_pool, block_table, seq_lens, max_seq_len: int, k_out=None, v_out=None,
                     stream=None):
    """The values the 4-bit cache holds, in logical order: k_out, v_out
    [S,Hkv,max_seq_len,D] bf16 (rows past a request's length are left as they were)."""
    if _torch is None:
        _load_torch()
    if _quick is not None and stream is None:
        r = _quick.gather(kv_pool, block_table, seq_lens, max_seq_len, k_out, v_out)
        if r is not None:
            return _done("paged_kv4_gather", r)
    _first(kv_pool)
    device = kv_pool.device
    NB = _check_kv4("kv_pool", kv_pool, None, None, device)
    _, Hkv, chunk = kv_pool.shape
    D = chunk // 18
    _check_tensor("seq_lens", seq_lens, _i32, None, device)
    if seq_lens.dim() != 1:
        raise ValueError("seq_lens must be a 1-d tensor")
    S, max_seq_len = seq_lens.shape[0], _length(max_seq_len)
    _check_table(block_table, S, device)
    shape = (S, Hkv, max_seq_len, D)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _check(name, t, _bf16, shape, device)
    _require_cuda(device)
    with _On(device, stream) as handle:
        if k_out is None:
            k_out = _torch.zeros(shape, dtype=_bf16, device=device)
        if v_out is None:
            v_out = _torch.zeros(shape, dtype=_bf16, device=device)
        st = (_lib or lib()).paged_kv4_gather(
            kv_pool.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), 16, S, Hkv, D,
            block_table.shape[1], NB, max_seq_len, k_out.data_ptr(), v_out.data_ptr(), handle)
    if st != ATTN_OK:
        raise GbAttnError("paged_kv4_gather", st)
    return k_out, v_out


def _length(n):
    """A bound on lengths as the C ABI's int."""
    n = int(n)
    if not 0 <= n < 1 << 31:
        raise ValueError(f"length bound out of range: {n}")
    return n


def _check_kv4_attention(q, kv_pool, block_table, lens, rows, out, lse):
    """The operands that the two attention calls share: q is [S, Hq, *rows, D]."""
    _first(q)
    device = q.device
    ndim = 3 + rows
    if q.dim() != ndim:
        raise ValueError(f"q must be a {ndim}-d tensor")
    shape = q.shape
    _check("q", q, _bf16, shape, device)
    NB = _check_kv4("kv_pool", kv_pool, None, None, device)
    _check_table(block_table, shape[0], device)
    _check("the lengths", lens, _i32, shape[:1], device)
    if kv_pool.shape[2] != 18 * shape[-1]:
        raise ValueError("inconsistent paged attention shapes")
    if out is not None:
        _check("out", out, _bf16, shape, device)
    if lse is not None:
        _check("lse", lse, _f32, shape[:-1], device)
    _require_cuda(device)
    return device, NB


def paged_kv4_attn_decode_workspace_size(num_seqs: int, Hq: int, Hkv: int, D: int,
                                         max_seq_len: int) -> int:
    return (_lib or lib()).paged_kv4_attn_decode_workspace_size(num_seqs, Hq, Hkv, D, max_seq_len)


def paged_kv4_attn_decode(q, kv_pool, block_table, seq_lens, max_seq_len: int,
                          scale: float | None = None, out=None, lse=None, workspace=None,
                          return_lse: bool = True, stream=None):
    """Single-token decode against the 4-bit paged cache through the C ABI.

    q [S,Hq,D] bf16, kv_pool [NB,Hkv,18*D] uint8, block_table [S,max_blocks] int32,
    seq_lens [S] int32 (all CUDA) -> (o [S,Hq,D] bf16, lse [S,Hq] fp32).
    ``workspace`` (uint8 CUDA tensor) is allocated here when not given.
    """
    if _torch is None:
        _load_torch()
    if _quick is not None and stream is None:
        r = _quick.decode(q, kv_pool, block_table, seq_lens, max_seq_len, scale, out, lse,
                          workspace, return_lse)
        if r is not None:
            return _done("paged_kv4_attn_decode", r)
    device, NB = _check_kv4_attention(q, kv_pool, block_table, seq_lens, 0, out, lse)
    S, Hq, D = q.shape
    max_seq_len = _length(max_seq_len)
    if workspace is not None:
        _check_tensor("workspace", workspace, _u8, None, device)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    with _On(device, stream) as handle:
        if workspace is None:
            need = paged_kv4_attn_decode_workspace_size(S, Hq, kv_pool.shape[1], D, max_seq_len)
            if need:
                workspace = _torch.empty((need,), dtype=_u8, device=device)
        if out is None:
            out = _torch.empty((S, Hq, D), dtype=_bf16, device=device)
        if return_lse and lse is None:
            lse = _torch.empty((S, Hq), dtype=_f32, device=device)
        st = (_lib or lib()).paged_kv4_attn_decode(
            q.data_ptr(), kv_pool.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), 16, S,
            Hq, kv_pool.shape[1], D, block_table.shape[1], NB, max_seq_len, scale, out.data_ptr(),
            _ptr(lse), _ptr(workspace), workspace.numel() if workspace is not None else 0, handle)
    if st != ATTN_OK:
        raise GbAttnError("paged_kv4_attn_decode", st)
    return out, lse


def paged_kv4_attn_prefill_workspace_size(B: int, Hq: int, Hkv: int, Tq: int, D: int,
                                          max_kv_len: int) -> int:
    return (_lib or lib()).paged_kv4_attn_prefill_workspace_size(B, Hq, Hkv, Tq, D, max_kv_len)


def paged_kv4_attn_prefill(q, kv_pool, block_table, kv_lens, max_kv_len: int,
                           causal: bool = True, scale: float | None = None, out=None, lse=None,
                           workspace=None, return_lse: bool = True, stream=None):
    """Chunked prefill against the 4-bit paged cache through the C ABI.

    q [B,Hq,Tq,D] bf16 (the Tq newest tokens of each item), kv_pool [NB,Hkv,18*D]
    uint8, block_table [B,max_blocks] int32, kv_lens [B] int32 (all CUDA) -> (o
    [B,Hq,Tq,D] bf16, lse [B,Hq,Tq] fp32).  Query i of item b sits at logical
    position kv_lens[b] - Tq + i.  ``workspace`` (uint8 CUDA tensor, needed for short
    chunks) is allocated here when not given.
    """
    if _torch is None:
        _load_torch()
    if _quick is not None and stream is None:
        r = _quick.prefill(q, kv_pool, block_table, kv_lens, max_kv_len, scale, out, lse, workspace,
                           return_lse, causal)
        if r is not None:
            return _done("paged_kv4_attn_prefill", r)
    device, NB = _check_kv4_attention(q, kv_pool, block_table, kv_lens, 1, out, lse)
    B, Hq, Tq, D = q.shape
    Hkv, max_kv_len = kv_pool.shape[1], _length(max_kv_len)
    if workspace is not None:
        _check_tensor("workspace", workspace, _u8, None, device)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    with _On(device, stream) as handle:
        if workspace is None:
            need = paged_kv4_attn_prefill_workspace_size(B, Hq, Hkv, Tq, D, max_kv_len)
            if need:
                workspace = _torch.empty((need,), dtype=_u8, device=device)
        if out is None:
            out = _torch.empty((B, Hq, Tq, D), dtype=_bf16, device=device)
        if return_lse and lse is None:
            lse = _torch.empty((B, Hq, Tq), dtype=_f32, device=device)
        st = (_lib or lib()).paged_kv4_attn_prefill(
            q.data_ptr(), kv_pool.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(), 16, B,
            Hq, Hkv, Tq, D, block_table.shape[1], NB, max_kv_len, 1 if causal else 0, scale,
            out.data_ptr(), _ptr(lse), _ptr(workspace),
            workspace.numel() if workspace is not None else 0, handle)
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
