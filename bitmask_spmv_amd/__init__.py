"""bitmask_spmv_amd -- N:M bitmask sparse decode kernels for AMD MI355X (gfx950).

Thin Python binding over the C ABI of ``include/nm_spmv.h`` (``libnmspmv.so``, built
in-tree by ``bitmask_spmv_amd._build``).  Every function has the C entry point's name
and only marshals arguments: it checks dtypes, devices, shapes and strides of torch
tensors, passes their device pointers and the current HIP stream, and turns a
non-zero status into :class:`NmError`.  All arithmetic runs in the HIP kernels; there
is no CPU fallback, and importing this package fails loudly when the library has not
been built.

PyTorch is used only for device memory and streams.  ``masks`` are carried in int32
tensors that hold the raw uint32 mask words; bf16 tensors are passed as raw patterns.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

__all__ = [
    "NmError", "LIB_PATH", "lib", "nm_version", "nm_col_norm", "nm_prune_pack", "nm_spmv",
    "nm_spmv_workspace_bytes", "dense_gemv", "dense_gemv_workspace_bytes", "nm_unpack",
    "NM_PATTERNS", "nm_spmv_multi", "nm_spmv_multi_workspace_bytes", "dense_gemv_multi",
    "dense_gemv_multi_workspace_bytes", "NM_META_BITMASK", "NM_META_U8_OFFSET", "NM_META_I32_INDEX",
    "nm_meta_from_mask", "nm_spmv_meta", "nm_spmv_swiglu", "nm_spmv_swiglu_workspace_bytes", "dense_gemv_swiglu",
    "dense_gemv_swiglu_workspace_bytes", "nm_prune_pack_unstructured", "nm_spmv_unstructured",
    "nm_spmv_unstructured_workspace_bytes", "nm_unpack_unstructured", "nm_hessian", "nm_obs_inverse_factor",
    "nm_obs_inverse_factor_workspace_bytes", "nm_sparsegpt_prune_pack", "nm_sparsegpt_workspace_bytes",
    "nm_stream_read", "nm_stream_read_sink_words", "nm_spmv_plan", "nm_spmv_multi_plan", "NM_EPI_NONE",
    "NM_EPI_SWIGLU", "NM_KERNEL_WORD", "NM_KERNEL_TILE", "NM_KERNEL_WORD_HALF_ROWS", "NM_KERNEL_WORD_STRIPS",
    "nm_spmv_noalloc", "nm_kv4_page_bytes", "nm_kv4_append", "nm_kv4_unpack", "nm_kv4_attention",
    "nm_kv4_attention_workspace_bytes", "nm_kv_pages_workspace_bytes", "nm_kv_resize", "nm_kv_fork",
    "nm_kv_compact", "nm_kv_copy_pages",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnmspmv.so")
NM_PATTERNS = ((2, 4), (4, 8), (8, 16), (16, 32))
NM_META_BITMASK, NM_META_U8_OFFSET, NM_META_I32_INDEX = 0, 1, 2
NM_EPI_NONE, NM_EPI_SWIGLU = 0, 1
NM_KERNEL_WORD, NM_KERNEL_TILE, NM_KERNEL_WORD_HALF_ROWS, NM_KERNEL_WORD_STRIPS = 0, 1, 2, 3

_STATUS = {0: "NM_OK", 1: "NM_ERR_NULL", 2: "NM_ERR_SHAPE", 3: "NM_ERR_PATTERN", 4: "NM_ERR_ALIGN",
           5: "NM_ERR_WORKSPACE", 6: "NM_ERR_HIP"}


class NmError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_STATUS.get(status, status)}: {detail}")


class _SpmvMatrix(ctypes.Structure):
    _fields_ = [("masks", ctypes.c_void_p), ("values", ctypes.c_void_p), ("R", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class _LaunchPlan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("threads", ctypes.c_int), ("grid_x", ctypes.c_int),
                ("splits", ctypes.c_int), ("tiles_per_step", ctypes.c_int), ("x_steps_in_registers", ctypes.c_int),
                ("rows_per_group", ctypes.c_int), ("lds_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t)]


class _DenseMatrix(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("R", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(or python bitmask_spmv_amd/_build.py); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    i64, p, i32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.nm_status_str.argtypes, L.nm_status_str.restype = [i32], ctypes.c_char_p
    L.nm_last_error.argtypes, L.nm_last_error.restype = [], ctypes.c_char_p
    L.nm_version.argtypes, L.nm_version.restype = [], i32
    L.nm_col_norm.argtypes = [p, i64, i64, i64, p, p]
    L.nm_prune_pack.argtypes = [p, i64, i64, i64, p, i32, i32, p, p, p]
    L.nm_spmv_workspace_bytes.argtypes, L.nm_spmv_workspace_bytes.restype = [i64, i64, i32], sz
    L.nm_spmv.argtypes = [p, p, i64, i64, p, i64, i32, p, i64, p, sz, p]
    L.nm_spmv_noalloc.argtypes, L.nm_spmv_noalloc.restype = [p, p, i64, i64, p, i64, i32, p, i64, p], i32
    L.dense_gemv_workspace_bytes.argtypes, L.dense_gemv_workspace_bytes.restype = [i64, i64, i32], sz
    L.dense_gemv.argtypes = [p, i64, i64, i64, p, i64, i32, p, i64, p, sz, p]
    L.nm_unpack.argtypes = [p, p, i64, i64, p, i64, p]
    L.nm_meta_from_mask.argtypes = [p, i64, i64, i32, p, p]
    f64 = ctypes.c_double
    L.nm_hessian.argtypes = [p, i64, i64, i64, p, i64, p]
    L.nm_obs_inverse_factor_workspace_bytes.argtypes = [i64]
    L.nm_obs_inverse_factor_workspace_bytes.restype = sz
    L.nm_obs_inverse_factor.argtypes = [p, i64, i64, f64, p, i64, p, sz, p]
    L.nm_sparsegpt_workspace_bytes.argtypes = [i64, i64]
    L.nm_sparsegpt_workspace_bytes.restype = sz
    L.nm_sparsegpt_prune_pack.argtypes = [p, i64, i64, i64, p, i64, i32, i32, f64, p, p, p, sz, p]
    L.nm_prune_pack_unstructured.argtypes = [p, i64, i64, i64, p, p, p, p]
    L.nm_spmv_unstructured_workspace_bytes.argtypes = [i64, i64, i32]
    L.nm_spmv_unstructured_workspace_bytes.restype = sz
    L.nm_spmv_unstructured.argtypes = [p, p, i64, i64, p, i64, i32, p, i64, p, sz, p]
    L.nm_unpack_unstructured.argtypes = [p, p, i64, i64, p, i64, p]
    L.nm_spmv_swiglu_workspace_bytes.argtypes, L.nm_spmv_swiglu_workspace_bytes.restype = [i64, i64, i32], sz
    L.nm_spmv_swiglu.argtypes = [p, p, p, p, i64, i64, p, i64, i32, p, i64, p, sz, p]
    L.dense_gemv_swiglu_workspace_bytes.argtypes, L.dense_gemv_swiglu_workspace_bytes.restype = [i64, i64, i32], sz
    L.dense_gemv_swiglu.argtypes = [p, p, i64, i64, i64, p, i64, i32, p, i64, p, sz, p]
    L.nm_spmv_meta.argtypes = [p, i32, p, i64, i64, p, i64, i32, p, i64, p, sz, p]
    L.nm_spmv_multi_workspace_bytes.argtypes = [p, i32, i64, i32]
    L.nm_spmv_multi_workspace_bytes.restype = sz
    L.nm_spmv_multi.argtypes = [p, i32, i64, p, i64, i32, p, sz, p]
    L.dense_gemv_multi_workspace_bytes.argtypes = [p, i32, i64, i32]
    L.dense_gemv_multi_workspace_bytes.restype = sz
    L.dense_gemv_multi.argtypes = [p, i32, i64, p, i64, i32, p, sz, p]
    L.nm_stream_read_sink_words.argtypes, L.nm_stream_read_sink_words.restype = [sz], sz
    L.nm_stream_read.argtypes, L.nm_stream_read.restype = [p, sz, p, sz, p], i32
    L.nm_spmv_plan.argtypes, L.nm_spmv_plan.restype = [i64, i64, i32, i32, p], i32
    L.nm_spmv_multi_plan.argtypes, L.nm_spmv_multi_plan.restype = [p, i32, i64, i32, p], i32
    f32 = ctypes.c_float
    L.nm_kv4_page_bytes.argtypes, L.nm_kv4_page_bytes.restype = [i32, i32, i32], i64
    d = ctypes.c_char_p  # a descriptor struct, packed by the caller
    L.nm_kv4_append.argtypes = L.nm_kv4_unpack.argtypes = [d, d, d, p]
    L.nm_kv4_attention_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i64, i64]
    L.nm_kv4_attention_workspace_bytes.restype = sz
    L.nm_kv4_attention.argtypes = [d, d, i32, i64, f32, i64, d, p, i64, p, sz, p]
    L.nm_kv_pages_workspace_bytes.argtypes, L.nm_kv_pages_workspace_bytes.restype = [i64, i64, i64, i32], sz
    L.nm_kv_resize.argtypes = [d, p, p, p, p, sz, p]
    L.nm_kv_fork.argtypes = [d, p, p, i64, p, p, p, sz, p]
    L.nm_kv_compact.argtypes = [d, p, i64, p, p, sz, p]
    L.nm_kv_copy_pages.argtypes = [p, i64, i64, i64, i64, p, i64, p]
    for f in (L.nm_kv4_append, L.nm_kv4_unpack, L.nm_kv4_attention, L.nm_kv_resize, L.nm_kv_fork, L.nm_kv_compact,
              L.nm_kv_copy_pages):
        f.restype = i32
    for f in (L.nm_col_norm, L.nm_prune_pack, L.nm_spmv, L.dense_gemv, L.nm_unpack, L.nm_spmv_multi,
              L.dense_gemv_multi):
        f.restype = i32
    return L


lib = _load()


def _check(status: int):
    if status != 0:
        raise NmError(status, lib.nm_last_error().decode(errors="replace"))


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on a HIP device (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D (got shape {tuple(t.shape)})")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else t.shape[-1]


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def nm_version() -> int:
    return int(lib.nm_version())


def nm_col_norm(X: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """X: bf16 [T, K] calibration activations -> fp32 [K] column norms."""
    _dev(X, "X", torch.bfloat16, 2)
    T, K = X.shape
    if out is None:
        out = torch.empty(K, dtype=torch.float32, device=X.device)
    _dev(out, "out", torch.float32, 1)
    _check(lib.nm_col_norm(_ptr(X), T, K, _ld(X), _ptr(out), _stream(X)))
    return out


def nm_prune_pack(W: torch.Tensor, col_norm: torch.Tensor, N: int, M: int, masks: torch.Tensor | None = None,
                  values: torch.Tensor | None = None):
    """W: bf16 [R, K]; col_norm: fp32 [K] -> (masks int32 [R, K/32], values bf16 [R, K/2])."""
    _dev(W, "W", torch.bfloat16, 2)
    _dev(col_norm, "col_norm", torch.float32, 1)
    R, K = W.shape
    if col_norm.shape[0] != K:
        raise ValueError("col_norm must have K entries")
    if masks is None:
        masks = torch.empty((R, max(K // 32, 1)), dtype=torch.int32, device=W.device)
    if values is None:
        values = torch.empty((R, max(K // 2, 1)), dtype=torch.bfloat16, device=W.device)
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    if not (masks.is_contiguous() and values.is_contiguous()):
        raise ValueError("masks and values must be contiguous")
    if K % 32 == 0 and (masks.shape != (R, K // 32) or values.shape != (R, K // 2)):
        raise ValueError("masks must be [R, K/32] and values [R, K/2]")
    _check(lib.nm_prune_pack(_ptr(W), _ld(W), R, K, _ptr(col_norm), int(N), int(M), _ptr(masks), _ptr(values),
                             _stream(W)))
    return masks, values


def nm_spmv_workspace_bytes(R: int, K: int, B: int) -> int:
    return int(lib.nm_spmv_workspace_bytes(R, K, B))


def dense_gemv_workspace_bytes(R: int, K: int, B: int) -> int:
    return int(lib.dense_gemv_workspace_bytes(R, K, B))


def _workspace(nbytes: int, ref: torch.Tensor, workspace: torch.Tensor | None):
    if nbytes == 0:
        return workspace, 0
    if workspace is None:
        workspace = torch.empty((nbytes + 3) // 4, dtype=torch.float32, device=ref.device)
    if workspace.device != ref.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    return workspace, workspace.numel() * workspace.element_size()


def _x_y(x: torch.Tensor, R: int, K: int, out: torch.Tensor | None):
    squeeze = x.dim() == 1
    if squeeze:
        x = x.unsqueeze(0)
    _dev(x, "x", torch.bfloat16, 2)
    B = x.shape[0]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} columns, expected K={K}")
    if out is None:
        out = torch.empty((B, R), dtype=torch.bfloat16, device=x.device)
    o2 = out.unsqueeze(0) if out.dim() == 1 else out
    _dev(o2, "out", torch.bfloat16, 2)
    if o2.shape != (B, R):
        raise ValueError(f"out must be [{B}, {R}]")
    return x, B, o2, out, squeeze


def nm_spmv(masks: torch.Tensor, values: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = W_sparse x for packed (masks, values); x: bf16 [B, K] or [K] -> bf16 [B, R] (or [R])."""
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    if not (masks.is_contiguous() and values.is_contiguous()):
        raise ValueError("masks and values must be contiguous")
    R = masks.shape[0]
    K = masks.shape[1] * 32
    if values.shape != (R, K // 2):
        raise ValueError("values must be [R, K/2] with K = 32 * masks.shape[1]")
    x2, B, o2, out, squeeze = _x_y(x, R, K, out)
    ws, ws_bytes = _workspace(nm_spmv_workspace_bytes(R, K, B), x2, workspace)
    _check(lib.nm_spmv(_ptr(masks), _ptr(values), R, K, _ptr(x2), _ld(x2), B, _ptr(o2), _ld(o2), _ptr(ws),
                       ws_bytes, _stream(x2)))
    return out[0] if squeeze and out.dim() == 2 else out


def nm_spmv_noalloc(masks: torch.Tensor, values: torch.Tensor, x: torch.Tensor,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """nm_spmv without a workspace: split rows use the library's fixed per-device scratch.
    Allocates nothing when `out` is given."""
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    if not (masks.is_contiguous() and values.is_contiguous()):
        raise ValueError("masks and values must be contiguous")
    R = masks.shape[0]
    K = masks.shape[1] * 32
    if values.shape != (R, K // 2):
        raise ValueError("values must be [R, K/2] with K = 32 * masks.shape[1]")
    x2, B, o2, out, squeeze = _x_y(x, R, K, out)
    _check(lib.nm_spmv_noalloc(_ptr(masks), _ptr(values), R, K, _ptr(x2), _ld(x2), B, _ptr(o2), _ld(o2),
                               _stream(x2)))
    return out[0] if squeeze and out.dim() == 2 else out


def dense_gemv(W: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = W x; W: bf16 [R, K]; x: bf16 [B, K] or [K] -> bf16 [B, R] (or [R])."""
    _dev(W, "W", torch.bfloat16, 2)
    R, K = W.shape
    x2, B, o2, out, squeeze = _x_y(x, R, K, out)
    ws, ws_bytes = _workspace(dense_gemv_workspace_bytes(R, K, B), x2, workspace)
    _check(lib.dense_gemv(_ptr(W), _ld(W), R, K, _ptr(x2), _ld(x2), B, _ptr(o2), _ld(o2), _ptr(ws), ws_bytes,
                          _stream(x2)))
    return out[0] if squeeze and out.dim() == 2 else out


def nm_unpack(masks: torch.Tensor, values: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Packed (masks, values) -> dense pruned bf16 [R, K] (zeros where bits are clear)."""
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    R = masks.shape[0]
    K = masks.shape[1] * 32
    if out is None:
        out = torch.empty((R, K), dtype=torch.bfloat16, device=masks.device)
    _dev(out, "out", torch.bfloat16, 2)
    _check(lib.nm_unpack(_ptr(masks), _ptr(values), R, K, _ptr(out), _ld(out), _stream(masks)))
    return out


def _meta_shape(fmt: int, R: int, K: int):
    if fmt == NM_META_BITMASK:
        return torch.int32, (R, K // 32)
    if fmt == NM_META_U8_OFFSET:
        return torch.uint8, (R, K // 2)
    if fmt == NM_META_I32_INDEX:
        return torch.int32, (R, K // 2)
    raise ValueError(f"unknown metadata format {fmt}")


def nm_meta_from_mask(masks: torch.Tensor, fmt: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Canonical masks int32 [R, K/32] -> uint8 offsets [R, K/2] (NM_META_U8_OFFSET) or int32
    column indices [R, K/2] (NM_META_I32_INDEX), in the order of the packed values."""
    _dev(masks, "masks", torch.int32, 2)
    if not masks.is_contiguous():
        raise ValueError("masks must be contiguous")
    R, K = masks.shape[0], masks.shape[1] * 32
    if fmt not in (NM_META_U8_OFFSET, NM_META_I32_INDEX):
        raise ValueError("fmt must be NM_META_U8_OFFSET or NM_META_I32_INDEX")
    dtype, shape = _meta_shape(fmt, R, K)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=masks.device)
    _dev(out, "out", dtype, 2)
    if out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {shape}")
    _check(lib.nm_meta_from_mask(_ptr(masks), R, K, int(fmt), _ptr(out), _stream(masks)))
    return out


def nm_spmv_meta(meta: torch.Tensor, fmt: int, values: torch.Tensor, x: torch.Tensor,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """nm_spmv with metadata in any format: masks int32 [R, K/32] (NM_META_BITMASK), uint8 offsets
    [R, K/2] (NM_META_U8_OFFSET) or int32 column indices [R, K/2] (NM_META_I32_INDEX)."""
    _dev(values, "values", torch.bfloat16, 2)
    R, K = values.shape[0], values.shape[1] * 2
    dtype, shape = _meta_shape(fmt, R, K)
    _dev(meta, "meta", dtype, 2)
    if meta.shape != shape or not (meta.is_contiguous() and values.is_contiguous()):
        raise ValueError(f"meta must be a contiguous {dtype} tensor of shape {shape}, values contiguous")
    x2, B, o2, out, squeeze = _x_y(x, R, K, out)
    ws, ws_bytes = _workspace(nm_spmv_workspace_bytes(R, K, B), x2, workspace)
    _check(lib.nm_spmv_meta(_ptr(meta), int(fmt), _ptr(values), R, K, _ptr(x2), _ld(x2), B, _ptr(o2), _ld(o2),
                            _ptr(ws), ws_bytes, _stream(x2)))
    return out[0] if squeeze and out.dim() == 2 else out


def nm_spmv_swiglu_workspace_bytes(R: int, K: int, B: int) -> int:
    return int(lib.nm_spmv_swiglu_workspace_bytes(R, K, B))


def dense_gemv_swiglu_workspace_bytes(R: int, K: int, B: int) -> int:
    return int(lib.dense_gemv_swiglu_workspace_bytes(R, K, B))


def nm_spmv_swiglu(gate, up, x: torch.Tensor, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """h = silu(W_gate x) * (W_up x) for packed gate = (masks, values) and up = (masks, values),
    both R x K; x: bf16 [B, K] or [K] -> bf16 [B, R] (or [R])."""
    (gm, gv), (um, uv) = gate, up
    for t, n, dt in ((gm, "gate masks", torch.int32), (gv, "gate values", torch.bfloat16),
                     (um, "up masks", torch.int32), (uv, "up values", torch.bfloat16)):
        _dev(t, n, dt, 2)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    R, K = gm.shape[0], gm.shape[1] * 32
    if gv.shape != (R, K // 2) or um.shape != gm.shape or uv.shape != gv.shape:
        raise ValueError("gate and up must both be packed R x K matrices")
    x2, B, o2, out, squeeze = _x_y(x, R, K, out)
    ws, ws_bytes = _workspace(nm_spmv_swiglu_workspace_bytes(R, K, B), x2, workspace)
    _check(lib.nm_spmv_swiglu(_ptr(gm), _ptr(gv), _ptr(um), _ptr(uv), R, K, _ptr(x2), _ld(x2), B, _ptr(o2),
                              _ld(o2), _ptr(ws), ws_bytes, _stream(x2)))
    return out[0] if squeeze and out.dim() == 2 else out


def dense_gemv_swiglu(W_gate: torch.Tensor, W_up: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Dense baseline of nm_spmv_swiglu: W_gate, W_up bf16 [R, K] with the same row stride."""
    _dev(W_gate, "W_gate", torch.bfloat16, 2)
    _dev(W_up, "W_up", torch.bfloat16, 2)
    if W_gate.shape != W_up.shape or _ld(W_gate) != _ld(W_up):
        raise ValueError("W_gate and W_up must have the same shape and row stride")
    R, K = W_gate.shape
    x2, B, o2, out, squeeze = _x_y(x, R, K, out)
    ws, ws_bytes = _workspace(dense_gemv_swiglu_workspace_bytes(R, K, B), x2, workspace)
    _check(lib.dense_gemv_swiglu(_ptr(W_gate), _ptr(W_up), _ld(W_gate), R, K, _ptr(x2), _ld(x2), B, _ptr(o2),
                                 _ld(o2), _ptr(ws), ws_bytes, _stream(x2)))
    return out[0] if squeeze and out.dim() == 2 else out


def nm_prune_pack_unstructured(W: torch.Tensor, col_norm: torch.Tensor, masks: torch.Tensor | None = None,
                               values: torch.Tensor | None = None):
    """50% unstructured: W bf16 [R, K], col_norm fp32 [K] -> (masks int32 [R, K/32], values bf16 [R, K/2]),
    each row keeping its K/2 highest scores."""
    _dev(W, "W", torch.bfloat16, 2)
    _dev(col_norm, "col_norm", torch.float32, 1)
    R, K = W.shape
    if col_norm.shape[0] != K:
        raise ValueError("col_norm must have K entries")
    if masks is None:
        masks = torch.empty((R, max(K // 32, 1)), dtype=torch.int32, device=W.device)
    if values is None:
        values = torch.empty((R, max(K // 2, 1)), dtype=torch.bfloat16, device=W.device)
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    if not (masks.is_contiguous() and values.is_contiguous()):
        raise ValueError("masks and values must be contiguous")
    if K % 32 == 0 and (masks.shape != (R, K // 32) or values.shape != (R, K // 2)):
        raise ValueError("masks must be [R, K/32] and values [R, K/2]")
    _check(lib.nm_prune_pack_unstructured(_ptr(W), _ld(W), R, K, _ptr(col_norm), _ptr(masks), _ptr(values),
                                          _stream(W)))
    return masks, values


def nm_spmv_unstructured_workspace_bytes(R: int, K: int, B: int) -> int:
    return int(lib.nm_spmv_unstructured_workspace_bytes(R, K, B))


def nm_spmv_unstructured(masks: torch.Tensor, values: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = W_sparse x for 50% unstructured rows packed by nm_prune_pack_unstructured."""
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    if not (masks.is_contiguous() and values.is_contiguous()):
        raise ValueError("masks and values must be contiguous")
    R, K = masks.shape[0], masks.shape[1] * 32
    if values.shape != (R, K // 2):
        raise ValueError("values must be [R, K/2] with K = 32 * masks.shape[1]")
    x2, B, o2, out, squeeze = _x_y(x, R, K, out)
    ws, ws_bytes = _workspace(nm_spmv_unstructured_workspace_bytes(R, K, B), x2, workspace)
    _check(lib.nm_spmv_unstructured(_ptr(masks), _ptr(values), R, K, _ptr(x2), _ld(x2), B, _ptr(o2), _ld(o2),
                                    _ptr(ws), ws_bytes, _stream(x2)))
    return out[0] if squeeze and out.dim() == 2 else out


def nm_unpack_unstructured(masks: torch.Tensor, values: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    R, K = masks.shape[0], masks.shape[1] * 32
    if out is None:
        out = torch.empty((R, K), dtype=torch.bfloat16, device=masks.device)
    _dev(out, "out", torch.bfloat16, 2)
    _check(lib.nm_unpack_unstructured(_ptr(masks), _ptr(values), R, K, _ptr(out), _ld(out), _stream(masks)))
    return out


def nm_hessian(X: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """H = 2 X^T X: X bf16 [T, K] calibration activations -> fp64 [K, K]."""
    _dev(X, "X", torch.bfloat16, 2)
    T, K = X.shape
    if out is None:
        out = torch.empty((K, K), dtype=torch.float64, device=X.device)
    _dev(out, "out", torch.float64, 2)
    if out.shape != (K, K):
        raise ValueError("out must be [K, K]")
    _check(lib.nm_hessian(_ptr(X), T, K, _ld(X), _ptr(out), _ld(out), _stream(X)))
    return out


def nm_obs_inverse_factor_workspace_bytes(K: int) -> int:
    return int(lib.nm_obs_inverse_factor_workspace_bytes(K))


def nm_obs_inverse_factor(H: torch.Tensor, damp: float = 0.01, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Upper U with U^T U = (H + damp * mean(diag H) * I)^-1 (fp64 [K, K])."""
    _dev(H, "H", torch.float64, 2)
    K = H.shape[0]
    if H.shape != (K, K):
        raise ValueError("H must be square")
    if out is None:
        out = torch.empty((K, K), dtype=torch.float64, device=H.device)
    _dev(out, "out", torch.float64, 2)
    ws, ws_bytes = _workspace(nm_obs_inverse_factor_workspace_bytes(K), H, workspace)
    _check(lib.nm_obs_inverse_factor(_ptr(H), _ld(H), K, float(damp), _ptr(out), _ld(out), _ptr(ws), ws_bytes,
                                     _stream(H)))
    return out


def nm_sparsegpt_workspace_bytes(R: int, K: int) -> int:
    return int(lib.nm_sparsegpt_workspace_bytes(R, K))


def nm_sparsegpt_prune_pack(W: torch.Tensor, H: torch.Tensor, N: int, M: int, damp: float = 0.01,
                            masks: torch.Tensor | None = None, values: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None):
    """OBS / SparseGPT N:M solver: W bf16 [R, K], H fp64 [K, K] -> (masks int32 [R, K/32], values bf16 [R, K/2])."""
    _dev(W, "W", torch.bfloat16, 2)
    _dev(H, "H", torch.float64, 2)
    R, K = W.shape
    if H.shape != (K, K):
        raise ValueError("H must be [K, K]")
    if masks is None:
        masks = torch.empty((R, max(K // 32, 1)), dtype=torch.int32, device=W.device)
    if values is None:
        values = torch.empty((R, max(K // 2, 1)), dtype=torch.bfloat16, device=W.device)
    _dev(masks, "masks", torch.int32, 2)
    _dev(values, "values", torch.bfloat16, 2)
    ws, ws_bytes = _workspace(nm_sparsegpt_workspace_bytes(R, K), W, workspace)
    _check(lib.nm_sparsegpt_prune_pack(_ptr(W), _ld(W), R, K, _ptr(H), _ld(H), int(N), int(M), float(damp),
                                       _ptr(masks), _ptr(values), _ptr(ws), ws_bytes, _stream(W)))
    return masks, values


def _multi_outs(x2, Rs, outs):
    B = x2.shape[0]
    if outs is None:
        outs = [torch.empty((B, R), dtype=torch.bfloat16, device=x2.device) for R in Rs]
    if len(outs) != len(Rs):
        raise ValueError("one output per matrix")
    o2 = []
    for o, R in zip(outs, Rs):
        o = o.unsqueeze(0) if o.dim() == 1 else o
        _dev(o, "out", torch.bfloat16, 2)
        if o.shape != (B, R):
            raise ValueError(f"out must be [{B}, {R}]")
        o2.append(o)
    return outs, o2


def _multi_x(x):
    x2 = x.unsqueeze(0) if x.dim() == 1 else x
    _dev(x2, "x", torch.bfloat16, 2)
    return x2


def nm_spmv_multi_workspace_bytes(Rs, K: int, B: int) -> int:
    arr = (_SpmvMatrix * len(Rs))(*[_SpmvMatrix(None, None, int(R), None, int(R)) for R in Rs])
    return int(lib.nm_spmv_multi_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(Rs), K, B))


def nm_spmv_multi(packed, x: torch.Tensor, outs=None, workspace: torch.Tensor | None = None):
    """Several packed matrices [(masks, values), ...] sharing x, in one launch -> list of y."""
    x2 = _multi_x(x)
    K = x2.shape[1]
    Rs = []
    for i, (m, v) in enumerate(packed):
        _dev(m, f"masks[{i}]", torch.int32, 2)
        _dev(v, f"values[{i}]", torch.bfloat16, 2)
        if not (m.is_contiguous() and v.is_contiguous()):
            raise ValueError("masks and values must be contiguous")
        if m.shape[1] * 32 != K or v.shape != (m.shape[0], K // 2):
            raise ValueError(f"matrix {i} does not have K={K} columns")
        Rs.append(m.shape[0])
    outs, o2 = _multi_outs(x2, Rs, outs)
    arr = (_SpmvMatrix * len(Rs))(*[_SpmvMatrix(m.data_ptr(), v.data_ptr(), R, o.data_ptr(), _ld(o))
                                     for (m, v), R, o in zip(packed, Rs, o2)])
    ws, ws_bytes = _workspace(int(lib.nm_spmv_multi_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(Rs), K,
                                                                     x2.shape[0])), x2, workspace)
    _check(lib.nm_spmv_multi(ctypes.cast(arr, ctypes.c_void_p), len(Rs), K, _ptr(x2), _ld(x2), x2.shape[0], _ptr(ws),
                             ws_bytes, _stream(x2)))
    return outs


def dense_gemv_multi_workspace_bytes(Rs, K: int, B: int) -> int:
    arr = (_DenseMatrix * len(Rs))(*[_DenseMatrix(None, K, int(R), None, int(R)) for R in Rs])
    return int(lib.dense_gemv_multi_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(Rs), K, B))


def dense_gemv_multi(Ws, x: torch.Tensor, outs=None, workspace: torch.Tensor | None = None):
    """Several dense matrices sharing x, in one launch -> list of y."""
    x2 = _multi_x(x)
    K = x2.shape[1]
    for i, W in enumerate(Ws):
        _dev(W, f"W[{i}]", torch.bfloat16, 2)
        if W.shape[1] != K:
            raise ValueError(f"matrix {i} does not have K={K} columns")
    Rs = [W.shape[0] for W in Ws]
    outs, o2 = _multi_outs(x2, Rs, outs)
    arr = (_DenseMatrix * len(Rs))(*[_DenseMatrix(W.data_ptr(), _ld(W), R, o.data_ptr(), _ld(o))
                                     for W, R, o in zip(Ws, Rs, o2)])
    ws, ws_bytes = _workspace(int(lib.dense_gemv_multi_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(Rs),
                                                                       K, x2.shape[0])), x2, workspace)
    _check(lib.dense_gemv_multi(ctypes.cast(arr, ctypes.c_void_p), len(Rs), K, _ptr(x2), _ld(x2), x2.shape[0],
                                _ptr(ws), ws_bytes, _stream(x2)))
    return outs


def nm_stream_read_sink_words(nbytes: int) -> int:
    return int(lib.nm_stream_read_sink_words(nbytes))


def nm_stream_read(buf: torch.Tensor, sink: torch.Tensor | None = None) -> torch.Tensor:
    """Measurement aid: one streaming read of a contiguous device tensor (its whole
    storage, a multiple of 16 bytes); returns the per-workgroup XOR folds (int32) whose
    XOR is the XOR of all dwords read."""
    if not isinstance(buf, torch.Tensor) or buf.device.type != "cuda":
        raise ValueError("buf must be a tensor on a HIP device")
    if not buf.is_contiguous():
        raise ValueError("buf must be contiguous")
    nbytes = buf.numel() * buf.element_size()
    words = nm_stream_read_sink_words(nbytes)
    if sink is None:
        sink = torch.empty(words, dtype=torch.int32, device=buf.device)
    _dev(sink, "sink", torch.int32, 1)
    _check(lib.nm_stream_read(_ptr(buf), nbytes, _ptr(sink), sink.numel(), _stream(buf)))
    return sink


def _plan_dict(pl: _LaunchPlan) -> dict:
    return {f: getattr(pl, f) for f, _ in _LaunchPlan._fields_}


def nm_spmv_plan(R: int, K: int, B: int, epilogue: int = NM_EPI_NONE) -> dict:
    """Launch plan of nm_spmv (or nm_spmv_swiglu with epilogue=NM_EPI_SWIGLU, R rows each)
    on the current device: kernel, threads, grid_x, splits, tiles_per_step,
    x_steps_in_registers, rows_per_group, lds_bytes, workspace_bytes.  Host only."""
    pl = _LaunchPlan()
    _check(lib.nm_spmv_plan(int(R), int(K), int(B), int(epilogue), ctypes.byref(pl)))
    return _plan_dict(pl)


def nm_spmv_multi_plan(rows, K: int, B: int) -> dict:
    """Launch plan of nm_spmv_multi over matrices with the given row counts.  Host only."""
    arr = (ctypes.c_int64 * len(rows))(*[int(r) for r in rows])
    pl = _LaunchPlan()
    _check(lib.nm_spmv_multi_plan(arr, len(rows), int(K), int(B), ctypes.byref(pl)))
    return _plan_dict(pl)


# ---- the 4-bit key/value cache (format, places and rules: include/nm_spmv.h) ----
#
# These run once a token and layer, some for a few microseconds: descriptors are packed in one
# go (native alignment, the C structs' field order), devices compared by number.

_KV4_BATCH = struct.Struct("@PqPqPPqq4i")  # nm_kv4_batch
_KV4_ROWS = struct.Struct("@Pqq")          # nm_kv4_rows
_KV_BOOK = struct.Struct("@PqPqPq2i")      # nm_kv_book


def nm_kv4_page_bytes(page_size: int, n_kv: int, head_dim: int) -> int:
    """Bytes of one page of page_size tokens (64, 128, 256 or 512) of n_kv heads of 64 or 128 channels."""
    return int(lib.nm_kv4_page_bytes(int(page_size), int(n_kv), int(head_dim)))


# The current stream's handle without the Python object around it (2 us of it), and the current device
# without the check that torch is initialised (a tensor on it is at hand), where torch has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_Tensor, _I32, _BF16 = torch.Tensor, torch.int32, torch.bfloat16


def _call(dev: int, fn, *args):
    """One entry point on device `dev`, on the stream that is current there."""
    stream = _raw_stream(dev)
    if dev == _current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status)


def _where(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a tensor on a HIP device")
    return t.get_device()


def _i32(t: torch.Tensor, name: str, dev: int, shape: tuple) -> int:
    if not isinstance(t, _Tensor) or t.dtype is not _I32 or t.get_device() != dev:
        raise TypeError(f"{name} must be an int32 tensor on cuda:{dev}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {list(shape)} (got {list(t.shape)})")
    return t.data_ptr()


def _table(t: torch.Tensor, dev: int):
    if not isinstance(t, _Tensor) or t.dtype is not _I32 or t.get_device() != dev:
        raise TypeError(f"page_table must be an int32 tensor on cuda:{dev}")
    stride = t.stride()
    if len(stride) != 2 or stride[1] != 1:
        raise ValueError("page_table must be [S, columns], contiguous in its last dimension")
    S, cols = t.shape
    return t.data_ptr(), stride[0] if S > 1 else cols, cols, S


def _kv_rows(t: torch.Tensor, name: str, dev: int, shape) -> bytes:
    if not isinstance(t, _Tensor) or t.dtype is not _BF16:
        raise TypeError(f"{name} must be a {torch.bfloat16} tensor")
    if t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must be on cuda:{dev}, of shape {list(shape)} (got {t.device}, {list(t.shape)})")
    stride = t.stride()
    if len(stride) != 3:
        raise ValueError(f"{name} must be [T, heads, head_dim]")
    ld, hd, one = stride
    if one != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    T, H, D = shape
    return _KV4_ROWS.pack(t.data_ptr(), ld if T > 1 else H * D, hd if H > 1 else D)


def _kv_batch(dev: int, cache: torch.Tensor, page_table, kv_len, q_start, page_size: int, n_kv: int, T: int, D: int):
    """(nm_kv4_batch, S, tokens a table row has room for), checked."""
    if not isinstance(cache, _Tensor) or cache.dtype is not torch.uint8 or cache.get_device() != dev:
        raise TypeError(f"cache must be a uint8 tensor on cuda:{dev}")
    if cache.dim() != 2 or not cache.is_contiguous():
        raise ValueError("cache must be contiguous, [num_pages, page_bytes]")
    N, nbytes = cache.shape
    if nbytes != page_size * n_kv * (D + D // 16):  # nm_kv4_page_bytes, where it is not 0
        raise ValueError(f"cache pages of {page_size} tokens of {n_kv} heads of {D} cannot have {nbytes} bytes")
    tp, ld, cols, S = _table(page_table, dev)
    return _KV4_BATCH.pack(cache.data_ptr(), N, tp, ld, _i32(kv_len, "kv_len", dev, (S,)),
                           _i32(q_start, "q_start", dev, (S + 1,)), S, T, cols, page_size, n_kv, D), S, cols * page_size


# Bytes that a call of some sizes on device `dev` needs: a function of them alone, asked once a size (1 us), with
# that device the current one (attention's depends on its compute units).
@functools.lru_cache(maxsize=4096)
def _attention_workspace(dev: int, *sizes) -> int:
    if dev == _current_device():
        return int(lib.nm_kv4_attention_workspace_bytes(*sizes))
    with torch.cuda.device(dev):
        return int(lib.nm_kv4_attention_workspace_bytes(*sizes))


@functools.lru_cache(maxsize=4096)
def _pages_workspace(dev: int, *sizes) -> int:
    return int(lib.nm_kv_pages_workspace_bytes(*sizes))


def _kv_workspace(query, dev: int, sizes: tuple, workspace: torch.Tensor | None):
    """(tensor to hold on to, pointer, bytes).  A workspace that is given is checked by the call itself."""
    if workspace is None:
        nbytes = query(dev, *sizes)
        if nbytes == 0:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
        return workspace, workspace.data_ptr(), nbytes
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def nm_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
                  kv_len: torch.Tensor, q_start: torch.Tensor, page_size: int) -> None:
    """Rows k, v bf16 [T, n_kv, D] -> cache uint8 [num_pages, page_bytes], at the last places of the
    sequences: page_table int32 [S, columns], kv_len int32 [S] (new rows included), q_start int32 [S + 1]."""
    dev, shape = _where(k, "k"), k.shape
    kr, vr = _kv_rows(k, "k", dev, shape), _kv_rows(v, "v", dev, shape)
    T, H, D = shape
    b, _, _ = _kv_batch(dev, cache, page_table, kv_len, q_start, page_size, H, T, D)
    _call(dev, lib.nm_kv4_append, b, kr, vr)


def nm_kv4_unpack(cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor,
                  page_size: int, k_out: torch.Tensor, v_out: torch.Tensor):
    """The rows that nm_kv4_append with the same arguments stores, as the cache holds them -> k_out, v_out bf16
    [T, n_kv, D]."""
    dev, shape = _where(k_out, "k_out"), k_out.shape
    kr, vr = _kv_rows(k_out, "k_out", dev, shape), _kv_rows(v_out, "v_out", dev, shape)
    T, H, D = shape
    b, _, _ = _kv_batch(dev, cache, page_table, kv_len, q_start, page_size, H, T, D)
    _call(dev, lib.nm_kv4_unpack, b, kr, vr)
    return k_out, v_out


def nm_kv4_attention_workspace_bytes(T: int, S: int, n_heads: int, n_kv: int, head_dim: int, max_q_len: int,
                                     room: int) -> int:
    """For calls on the current device.  room: tokens that a row of the page table has room for (columns * page_size)."""
    return int(lib.nm_kv4_attention_workspace_bytes(T, S, n_heads, n_kv, head_dim, max_q_len, room))


def nm_kv4_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                     q_start: torch.Tensor, n_kv: int, page_size: int, max_q_len: int, scale: float | None = None,
                     window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """Causal attention of rows q bf16 [T, heads, D] over the cached keys and values of their sequences ->
    (out bf16 [T, heads, D], lse fp32 [T, heads]).  scale: 1 / sqrt(D) unless given.  window: keys a row looks
    back over, itself among them (0: all).  max_q_len: a hint, the most rows of one sequence."""
    dev, shape = _where(q, "q"), q.shape
    qr = _kv_rows(q, "q", dev, shape)
    T, Hq, D = shape
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    elif lse.dtype is not torch.float32 or lse.get_device() != dev or lse.shape != (T, Hq) or lse.stride(1) != 1:
        raise ValueError("lse must be fp32 [T, heads], contiguous in its last dimension, on q's device")
    b, S, room = _kv_batch(dev, cache, page_table, kv_len, q_start, page_size, n_kv, T, D)
    ws, wp, wn = _kv_workspace(_attention_workspace, dev, (T, S, Hq, n_kv, D, max_q_len, room), workspace)
    _call(dev, lib.nm_kv4_attention, b, qr, Hq, max_q_len, D ** -0.5 if scale is None else scale, window,
          _kv_rows(out, "out", dev, shape), lse.data_ptr(), lse.stride(0) if T > 1 else Hq, wp, wn)
    return out, lse


def nm_kv_pages_workspace_bytes(S: int, n_pairs: int, num_pages: int, table_cols: int) -> int:
    return int(lib.nm_kv_pages_workspace_bytes(S, n_pairs, num_pages, table_cols))


def _kv_book(dev: int, page_table, kv_len, refcount, page_size, n_pairs, workspace):
    """(nm_kv_book, S, workspace, its pointer and bytes), checked."""
    tp, ld, cols, S = _table(page_table, dev)
    N = refcount.numel()
    b = _KV_BOOK.pack(tp, ld, _i32(kv_len, "kv_len", dev, (S,)), S, _i32(refcount, "refcount", dev, (N,)), N, cols, page_size)
    return b, S, *_kv_workspace(_pages_workspace, dev, (S, n_pairs, N, cols), workspace)


def nm_kv_resize(new_len: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, refcount: torch.Tensor,
                 page_size: int, moves: torch.Tensor, missing: torch.Tensor,
                 workspace: torch.Tensor | None = None) -> None:
    """Sequences to new_len int32 [S] tokens: pages given back or handed out, in page_table int32 [S, columns],
    kv_len int32 [S] and refcount int32 [num_pages].  moves int32 [S, 2] for nm_kv_copy_pages; missing int32 [1]."""
    dev = _where(page_table, "page_table")
    b, S, ws, wp, wn = _kv_book(dev, page_table, kv_len, refcount, page_size, 0, workspace)
    _call(dev, lib.nm_kv_resize, b, _i32(new_len, "new_len", dev, (S,)), _i32(moves, "moves", dev, (S, 2)),
          _i32(missing, "missing", dev, (1,)), wp, wn)


def nm_kv_fork(parent: torch.Tensor, child: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
               refcount: torch.Tensor, page_size: int, moves: torch.Tensor, missing: torch.Tensor,
               workspace: torch.Tensor | None = None) -> None:
    """Slots child int32 [n] become copies of slots parent int32 [n]; full pages are shared.  moves int32 [n, 2]
    for nm_kv_copy_pages; missing int32 [1]."""
    dev, n = _where(page_table, "page_table"), parent.numel()
    b, S, ws, wp, wn = _kv_book(dev, page_table, kv_len, refcount, page_size, n, workspace)
    _call(dev, lib.nm_kv_fork, b, _i32(parent, "parent", dev, (n,)), _i32(child, "child", dev, (n,)), n,
          _i32(moves, "moves", dev, (n, 2)), _i32(missing, "missing", dev, (1,)), wp, wn)


def nm_kv_compact(page_table: torch.Tensor, kv_len: torch.Tensor, refcount: torch.Tensor, page_size: int,
                  moves: torch.Tensor, used: torch.Tensor, workspace: torch.Tensor | None = None) -> None:
    """Used pages into the lowest numbers.  moves int32 [max_moves, 2] for nm_kv_copy_pages; used int32 [1]."""
    dev, n = _where(page_table, "page_table"), moves.shape[0]
    b, S, ws, wp, wn = _kv_book(dev, page_table, kv_len, refcount, page_size, 0, workspace)
    _call(dev, lib.nm_kv_compact, b, _i32(moves, "moves", dev, (n, 2)), n, _i32(used, "used", dev, (1,)), wp, wn)


def nm_kv_copy_pages(cache: torch.Tensor, moves: torch.Tensor) -> None:
    """Copies page moves[i, 0] to page moves[i, 1] (int32 [n, 2]) of cache uint8 [num_pages, page_bytes], or in
    each layer of [layers, num_pages, page_bytes]."""
    dev = _where(cache, "cache")
    if cache.dtype is not torch.uint8 or cache.dim() not in (2, 3):
        raise TypeError("cache must be uint8 [num_pages, page_bytes] or [layers, num_pages, page_bytes]")
    N, nbytes = cache.shape[-2:]
    layers, stride = (cache.shape[0], cache.stride(0)) if cache.dim() == 3 else (1, N * nbytes)
    if cache.stride()[-2:] != (nbytes, 1):
        raise ValueError("the pages of a layer must be contiguous")
    n = moves.shape[0]
    _call(dev, lib.nm_kv_copy_pages, cache.data_ptr(), N, nbytes, layers, stride, _i32(moves, "moves", dev, (n, 2)), n)
