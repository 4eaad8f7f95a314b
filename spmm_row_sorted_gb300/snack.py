"""Thin Python binding of libsnack (include/snack.h).

The functions named ``snack_*`` mirror the C entry points one to one and only
marshal arguments: torch tensors become device pointers and byte sizes, the
stream defaults to torch's current stream.  Every computation runs in the CUDA
library; when the library has not been built, loading it raises
``SnackLibraryMissing`` -- there is no fallback of any kind.

``SparseLinear`` is a convenience owner of one layer (pattern, values, bias,
plan and workspace tensors) on top of those calls, and ``sparse_linear`` an
autograd function over it.
"""

from __future__ import annotations

import array
import ctypes
import functools
import os
import threading
from typing import Optional

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import build as _build

SNACK_OK = 0
STATUS_NAMES = {0: "SNACK_OK", 1: "SNACK_ERR_INVALID_ARG", 2: "SNACK_ERR_UNSORTED", 3: "SNACK_ERR_OUT_OF_RANGE",
                4: "SNACK_ERR_WORKSPACE", 5: "SNACK_ERR_CUDA", 6: "SNACK_ERR_TIMEOUT", 7: "SNACK_ERR_UNSUPPORTED",
                8: "SNACK_ERR_NO_SPACE"}
SNACK_F32, SNACK_BF16 = 0, 1
SNACK_I32, SNACK_I64 = 0, 1
REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}

EXPORTED = ("snack_query_sizes", "snack_create", "snack_spmm_fwd", "snack_spmm_fwd_noalloc", "snack_spmm_dx",
            "snack_spmm_fwd_gelu", "snack_spmm_dx_gelu", "snack_sddmm_dw", "snack_backward",
            "snack_restructure_workspace_size", "snack_restructure", "snack_restructure_rows_workspace_size",
            "snack_restructure_rows", "snack_wait_plan", "snack_destroy", "snack_status_string", "snack_version",
            "snack_trace_start", "snack_trace_read", "snack_trace_stop", "snack_embed_fwd",
            "snack_embed_grad_workspace_size", "snack_embed_grad", "snack_clip_workspace_size",
            "snack_clip_grad_norm", "snack_xent_workspace_size", "snack_xent_fwd", "snack_xent_bwd",
            "snack_adapt_workspace_size", "snack_adapt_fwd", "snack_adapt_bwd", "snack_score_workspace_size",
            "snack_score_fwd", "snack_score_bwd")


class SnackLibraryMissing(RuntimeError):
    pass


class SnackError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({msg})")
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(path: Optional[str] = None):
    """Load libsnack.so (must have been built with spmm_row_sorted_gb300.build.build())."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            raise SnackLibraryMissing(f"{p} is missing: build it with `python -m spmm_row_sorted_gb300.build`")
        lib = ctypes.CDLL(p)
        vp, i32, i64, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
        st = ctypes.c_int
        lib.snack_query_sizes.argtypes = [i32, i32, i64, i32, st, st, ctypes.POINTER(sz), ctypes.POINTER(sz)]
        lib.snack_query_sizes.restype = st
        lib.snack_create.argtypes = [ctypes.POINTER(vp), i32, i32, i64, i32, st, st, vp, vp, vp, sz, vp, sz,
                                     ctypes.c_int, vp]
        lib.snack_create.restype = st
        lib.snack_spmm_fwd.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
        lib.snack_spmm_fwd.restype = st
        lib.snack_spmm_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp]
        lib.snack_spmm_fwd_noalloc.restype = st
        lib.snack_spmm_fwd_gelu.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]
        lib.snack_spmm_fwd_gelu.restype = st
        lib.snack_spmm_dx_gelu.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
        lib.snack_spmm_dx_gelu.restype = st
        lib.snack_spmm_dx.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, sz, vp]
        lib.snack_spmm_dx.restype = st
        lib.snack_sddmm_dw.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
        lib.snack_sddmm_dw.restype = st
        lib.snack_backward.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]
        lib.snack_backward.restype = st
        lib.snack_restructure_workspace_size.argtypes = [vp, i64, ctypes.POINTER(sz)]
        lib.snack_restructure_workspace_size.restype = st
        lib.snack_restructure.argtypes = [vp, vp, vp, vp, i64, u64, u64, vp, vp, vp, vp, vp, sz, vp]
        lib.snack_restructure.restype = st
        lib.snack_restructure_rows_workspace_size.argtypes = [vp, i64, ctypes.POINTER(sz)]
        lib.snack_restructure_rows_workspace_size.restype = st
        lib.snack_restructure_rows.argtypes = [vp, vp, vp, vp, i64, u64, u64, vp, vp, vp, vp, vp, sz, vp]
        lib.snack_restructure_rows.restype = st
        lib.snack_wait_plan.argtypes = [vp, vp]
        lib.snack_wait_plan.restype = st
        lib.snack_destroy.argtypes = [vp]
        lib.snack_destroy.restype = None
        lib.snack_status_string.argtypes = [st]
        lib.snack_status_string.restype = ctypes.c_char_p
        lib.snack_version.argtypes = []
        lib.snack_version.restype = ctypes.c_int
        lib.snack_trace_start.argtypes = [i32]
        lib.snack_trace_start.restype = st
        lib.snack_trace_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float), i32,
                                         ctypes.POINTER(i32)]
        lib.snack_trace_read.restype = st
        lib.snack_trace_stop.argtypes = []
        lib.snack_trace_stop.restype = st
        f32 = ctypes.c_float
        lib.snack_embed_fwd.argtypes = [vp, st, i64, vp, i64, i64, i32, st, f32, vp, i64, vp]
        lib.snack_embed_fwd.restype = st
        lib.snack_embed_grad_workspace_size.argtypes = [i64, i64, i32, ctypes.POINTER(sz)]
        lib.snack_embed_grad_workspace_size.restype = st
        lib.snack_embed_grad.argtypes = [vp, st, i64, vp, i64, i64, i32, st, f32, ctypes.c_int, vp, i64, vp, sz, vp]
        lib.snack_embed_grad.restype = st
        lib.snack_clip_workspace_size.argtypes = [i32, vp, vp, ctypes.POINTER(sz)]
        lib.snack_clip_workspace_size.restype = st
        lib.snack_clip_grad_norm.argtypes = [i32, vp, vp, vp, vp, f32, vp, vp, sz, vp]
        lib.snack_clip_grad_norm.restype = st
        lib.snack_xent_workspace_size.argtypes = [vp, i64, i32, vp, i64, i64, i32, st, ctypes.c_int, ctypes.POINTER(sz)]
        lib.snack_xent_workspace_size.restype = st
        lib.snack_xent_fwd.argtypes = [vp, i64, i32, vp, i64, i64, i32, st, vp, st, st, vp, vp, vp, sz, vp]
        lib.snack_xent_fwd.restype = st
        lib.snack_xent_bwd.argtypes = [vp, i64, i32, vp, i64, i64, i32, st, vp, st, st, vp, vp, vp, i64, vp, i64, vp, sz,
                                       vp]
        lib.snack_xent_bwd.restype = st
        lib.snack_adapt_workspace_size.argtypes = [i64, i32, i32, ctypes.POINTER(sz)]
        lib.snack_adapt_workspace_size.restype = st
        lib.snack_adapt_fwd.argtypes = [vp, i64, i64, vp, vp, i32, i32, i32, i32, st, vp, st, vp, vp, i64, vp, i64, vp, vp,
                                        sz, vp]
        lib.snack_adapt_fwd.restype = st
        lib.snack_adapt_bwd.argtypes = [vp, i64, i64, vp, vp, i32, i32, i32, i32, st, vp, st, vp, vp, vp, i64, ctypes.c_int,
                                        vp, i64, vp, vp, vp, sz, vp]
        lib.snack_adapt_bwd.restype = st
        lib.snack_score_workspace_size.argtypes = [vp, i64, i32, vp, i64, i64, i32, st, i32, ctypes.c_int, ctypes.POINTER(sz)]
        lib.snack_score_workspace_size.restype = st
        lib.snack_score_fwd.argtypes = [vp, i64, i32, vp, i64, i64, i32, st, vp, st, vp, vp, i32, vp, vp, vp, vp, sz, vp]
        lib.snack_score_fwd.restype = st
        lib.snack_score_bwd.argtypes = [vp, i64, i32, vp, i64, i64, i32, st, vp, st, vp, vp, vp, vp, i64, vp, i64, vp, sz, vp]
        lib.snack_score_bwd.restype = st
        _lib = lib
        return lib


def _check(fn: str, status: int) -> None:
    if status:
        raise SnackError(fn, status, load().snack_status_string(status).decode())


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _raw_stream(stream):
    """The cudaStream_t of `stream`, or of torch's current one, as an integer."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return SNACK_F32
    if dt == torch.bfloat16:
        return SNACK_BF16
    raise ValueError(f"unsupported dtype {dt}")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


# ------------------------------------------------------------- raw entry points


def snack_query_sizes(out_f: int, in_f: int, nnz: int, max_batch: int, val_t: int, act_t: int):
    p, w = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("snack_query_sizes",
           load().snack_query_sizes(out_f, in_f, nnz, max_batch, val_t, act_t, ctypes.byref(p), ctypes.byref(w)))
    return p.value, w.value


def snack_create(out_f: int, in_f: int, nnz: int, max_batch: int, val_t: int, act_t: int, row, col,
                 plan: torch.Tensor, ws: torch.Tensor, validate: bool = False, stream=None) -> int:
    h = ctypes.c_void_p(0)
    _check("snack_create",
           load().snack_create(ctypes.byref(h), out_f, in_f, nnz, max_batch, val_t, act_t, _ptr(row), _ptr(col),
                               _ptr(plan), _nbytes(plan), _ptr(ws), _nbytes(ws), 1 if validate else 0,
                               _stream(stream)))
    return h.value


def snack_spmm_fwd(h: int, row, col, val, x, batch: int, bias, y, ws, stream=None) -> None:
    _check("snack_spmm_fwd",
           load().snack_spmm_fwd(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), _ptr(x), batch, _ptr(bias),
                                 _ptr(y), _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def snack_spmm_fwd_noalloc(h: int, row, col, val, x, batch: int, bias, y, stream=None) -> None:
    """Forward pass using the library's built-in scratch array (no workspace argument)."""
    _check("snack_spmm_fwd_noalloc",
           load().snack_spmm_fwd_noalloc(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), _ptr(x), batch,
                                         _ptr(bias), _ptr(y), _stream(stream)))


def snack_spmm_dx(h: int, row, col, val, dy, batch: int, dx, ws, stream=None) -> None:
    _check("snack_spmm_dx",
           load().snack_spmm_dx(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), _ptr(dy), batch, _ptr(dx),
                                _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def snack_spmm_fwd_gelu(h: int, row, col, val, x, batch: int, bias, y_pre, y, ws, stream=None) -> None:
    _check("snack_spmm_fwd_gelu",
           load().snack_spmm_fwd_gelu(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), _ptr(x), batch, _ptr(bias),
                                      _ptr(y_pre), _ptr(y), _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def snack_spmm_dx_gelu(h: int, row, col, val, dy, batch: int, x_pre, dx, ws, stream=None) -> None:
    _check("snack_spmm_dx_gelu",
           load().snack_spmm_dx_gelu(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), _ptr(dy), batch,
                                     _ptr(x_pre), _ptr(dx), _ptr(ws), 0 if ws is None else _nbytes(ws),
                                     _stream(stream)))


def snack_sddmm_dw(h: int, row, col, x, dy, batch: int, dw, db, ws, stream=None) -> None:
    _check("snack_sddmm_dw",
           load().snack_sddmm_dw(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(x), _ptr(dy), batch, _ptr(dw),
                                 _ptr(db), _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def snack_backward(h: int, row, col, val, x, dy, batch: int, dx, dw, db, ws, stream=None) -> None:
    _check("snack_backward",
           load().snack_backward(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), _ptr(x), _ptr(dy), batch,
                                 _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), 0 if ws is None else _nbytes(ws),
                                 _stream(stream)))


def snack_restructure_workspace_size(h: int, n_prune: int) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_restructure_workspace_size",
           load().snack_restructure_workspace_size(ctypes.c_void_p(h), n_prune, ctypes.byref(b)))
    return b.value


def snack_restructure(h: int, row, col, val, n_prune: int, seed: int, step: int, row_out, col_out, val_out,
                      src_out, ws, stream=None) -> None:
    _check("snack_restructure",
           load().snack_restructure(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), n_prune,
                                    seed & (2**64 - 1), step & (2**64 - 1), _ptr(row_out), _ptr(col_out),
                                    _ptr(val_out), _ptr(src_out), _ptr(ws), _nbytes(ws), _stream(stream)))


def snack_restructure_rows_workspace_size(h: int, n_per_row: int) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_restructure_rows_workspace_size",
           load().snack_restructure_rows_workspace_size(ctypes.c_void_p(h), n_per_row, ctypes.byref(b)))
    return b.value


def snack_restructure_rows(h: int, row, col, val, n_per_row: int, seed: int, step: int, row_out, col_out, val_out,
                           src_out, ws, stream=None) -> None:
    _check("snack_restructure_rows",
           load().snack_restructure_rows(ctypes.c_void_p(h), _ptr(row), _ptr(col), _ptr(val), n_per_row,
                                         seed & (2**64 - 1), step & (2**64 - 1), _ptr(row_out), _ptr(col_out),
                                         _ptr(val_out), _ptr(src_out), _ptr(ws), _nbytes(ws), _stream(stream)))


def snack_wait_plan(h: int, stream=None) -> None:
    _check("snack_wait_plan", load().snack_wait_plan(ctypes.c_void_p(h), _stream(stream)))


def snack_destroy(h: int) -> None:
    load().snack_destroy(ctypes.c_void_p(h))


def snack_status_string(status: int) -> str:
    return load().snack_status_string(status).decode()


def snack_trace_start(capacity: int) -> None:
    _check("snack_trace_start", load().snack_trace_start(capacity))


def snack_trace_read(max_records: int) -> list:
    """The last records of the calling thread's trace, oldest first: (kernel name, microseconds)."""
    names = (ctypes.c_char_p * max(max_records, 1))()
    us = (ctypes.c_float * max(max_records, 1))()
    n = ctypes.c_int32(0)
    _check("snack_trace_read", load().snack_trace_read(names, us, max_records, ctypes.byref(n)))
    return [(names[i].decode(), float(us[i])) for i in range(n.value)]


def snack_trace_stop() -> None:
    _check("snack_trace_stop", load().snack_trace_stop())


def snack_version() -> int:
    return int(load().snack_version())


def index_code(dt: torch.dtype) -> int:
    if dt == torch.int32:
        return SNACK_I32
    if dt == torch.int64:
        return SNACK_I64
    raise ValueError(f"unsupported index dtype {dt}")


def snack_embed_fwd(ids, table, scale: float, out, stream=None) -> None:
    _check("snack_embed_fwd",
           (_lib or load()).snack_embed_fwd(_addr(ids), index_code(ids.dtype), ids.numel(), _addr(table), table.stride(0),
                                  table.shape[0], table.shape[1], dtype_code(table.dtype), scale, _addr(out),
                                  out.stride(0), _raw_stream(stream)))


def snack_embed_grad_workspace_size(n: int, vocab: int, width: int) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_embed_grad_workspace_size",
           (_lib or load()).snack_embed_grad_workspace_size(n, vocab, width, ctypes.byref(b)))
    return b.value


def snack_embed_grad(ids, dout, scale: float, accumulate: bool, dtable, ws, stream=None) -> None:
    _check("snack_embed_grad",
           (_lib or load()).snack_embed_grad(_addr(ids), index_code(ids.dtype), ids.numel(), _addr(dout), dout.stride(0),
                                   dtable.shape[0], dtable.shape[1], dtype_code(dtable.dtype), scale,
                                   1 if accumulate else 0, _addr(dtable), dtable.stride(0), _addr(ws), _nbytes(ws),
                                   _raw_stream(stream)))


def snack_clip_workspace_size(numel, types) -> int:
    b = ctypes.c_size_t(0)
    m, t = _array("q", numel), _array("i", types)
    _check("snack_clip_workspace_size",
           load().snack_clip_workspace_size(len(numel), _at(m), _at(t), ctypes.byref(b)))
    return b.value


def _array(code: str, values) -> array.array:
    """`values` as a C array: "Q" addresses, "q" int64, "i" int."""
    return array.array(code, values)


def _at(a: array.array):
    return a.buffer_info()[0] if a else None


def snack_clip_grad_norm(grads, outs, numel, types, max_norm: float, norm, ws, stream=None) -> None:
    """grads and outs: lists of device addresses (outs None: the norm alone); numel, types: lists of their sizes."""
    if not len(grads) == len(numel) == len(types) or (outs is not None and len(outs) != len(grads)):
        raise ValueError("one address, size and type per tensor")
    g, o, m, t = (_array(c, v) for c, v in (("Q", grads), ("Q", outs or ()), ("q", numel), ("i", types)))
    _check("snack_clip_grad_norm",
           (_lib or load()).snack_clip_grad_norm(len(grads), _at(g), None if outs is None else _at(o), _at(m), _at(t),
                                                 max_norm, _addr(norm), _addr(ws), _nbytes(ws), _raw_stream(stream)))


def snack_xent_workspace_size(x, w, grad: bool) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_xent_workspace_size",
           (_lib or load()).snack_xent_workspace_size(_addr(x), x.stride(0), x.shape[0], _addr(w), w.stride(0), w.shape[0],
                                            w.shape[1], dtype_code(w.dtype), 1 if grad else 0, ctypes.byref(b)))
    return b.value


def snack_xent_fwd(x, w, targets, reduction: int, loss, state, ws, stream=None) -> None:
    _check("snack_xent_fwd",
           (_lib or load()).snack_xent_fwd(_addr(x), x.stride(0), x.shape[0], _addr(w), w.stride(0), w.shape[0], w.shape[1],
                                 dtype_code(w.dtype), _addr(targets), index_code(targets.dtype), reduction, _addr(loss),
                                 _addr(state), _addr(ws), _nbytes(ws), _raw_stream(stream)))


def snack_xent_bwd(x, w, targets, reduction: int, state, dloss, dx, dw, ws, stream=None) -> None:
    _check("snack_xent_bwd",
           (_lib or load()).snack_xent_bwd(_addr(x), x.stride(0), x.shape[0], _addr(w), w.stride(0), w.shape[0], w.shape[1],
                                 dtype_code(w.dtype), _addr(targets), index_code(targets.dtype), reduction, _addr(state),
                                 _addr(dloss), _addr(dx), 0 if dx is None else dx.stride(0), _addr(dw),
                                 0 if dw is None else dw.stride(0), _addr(ws), _nbytes(ws), _raw_stream(stream)))


def snack_adapt_workspace_size(n: int, n_adapters: int, rank: int) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_adapt_workspace_size",
           (_lib or load()).snack_adapt_workspace_size(n, n_adapters, rank, ctypes.byref(b)))
    return b.value


def snack_adapt_fwd(x, a, b, which, scales, base, y, h, ws, stream=None) -> None:
    _check("snack_adapt_fwd",
           (_lib or load()).snack_adapt_fwd(_addr(x), x.stride(0), x.shape[0], _addr(a), _addr(b), a.shape[0], a.shape[1],
                                            x.shape[1], y.shape[1], dtype_code(x.dtype), _addr(which),
                                            index_code(which.dtype), _addr(scales), _addr(base),
                                            0 if base is None else base.stride(0), _addr(y), y.stride(0), _addr(h),
                                            _addr(ws), _nbytes(ws), _raw_stream(stream)))


def snack_adapt_bwd(x, a, b, which, scales, h, dy, accumulate: bool, dx, da, db, ws, stream=None) -> None:
    _check("snack_adapt_bwd",
           (_lib or load()).snack_adapt_bwd(_addr(x), x.stride(0), x.shape[0], _addr(a), _addr(b), a.shape[0], a.shape[1],
                                            x.shape[1], dy.shape[1], dtype_code(x.dtype), _addr(which),
                                            index_code(which.dtype), _addr(scales), _addr(h), _addr(dy), dy.stride(0),
                                            1 if accumulate else 0, _addr(dx), 0 if dx is None else dx.stride(0),
                                            _addr(da), _addr(db), _addr(ws), _nbytes(ws), _raw_stream(stream)))


def snack_score_workspace_size(x, w, top: int, grad: bool) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_score_workspace_size",
           (_lib or load()).snack_score_workspace_size(_addr(x), x.stride(0), x.shape[0], _addr(w), w.stride(0), w.shape[0],
                                                       w.shape[1], dtype_code(w.dtype), top, 1 if grad else 0,
                                                       ctypes.byref(b)))
    return b.value


def snack_score_fwd(x, w, targets, logp, entropy, top: int, top_ids, top_logp, state, ws, stream=None) -> None:
    _check("snack_score_fwd",
           (_lib or load()).snack_score_fwd(_addr(x), x.stride(0), x.shape[0], _addr(w), w.stride(0), w.shape[0], w.shape[1],
                                            dtype_code(w.dtype), _addr(targets),
                                            SNACK_I64 if targets is None else index_code(targets.dtype), _addr(logp),
                                            _addr(entropy), top, _addr(top_ids), _addr(top_logp), _addr(state), _addr(ws),
                                            _nbytes(ws), _raw_stream(stream)))


def snack_score_bwd(x, w, targets, state, dlogp, dentropy, dx, dw, ws, stream=None) -> None:
    _check("snack_score_bwd",
           (_lib or load()).snack_score_bwd(_addr(x), x.stride(0), x.shape[0], _addr(w), w.stride(0), w.shape[0], w.shape[1],
                                            dtype_code(w.dtype), _addr(targets),
                                            SNACK_I64 if targets is None else index_code(targets.dtype), _addr(state),
                                            _addr(dlogp), _addr(dentropy), _addr(dx), 0 if dx is None else dx.stride(0),
                                            _addr(dw), 0 if dw is None else dw.stride(0), _addr(ws), _nbytes(ws),
                                            _raw_stream(stream)))


# ------------------------------------------------------------- layer owner


class SparseLinear:
    """One truly sparse layer on the GPU: Y = X W^T + b over the stored weights.

    row/col: int32 CUDA tensors (row-sorted COO, strictly increasing in
    (row, col)); val: float32 or bfloat16 CUDA tensor; bias: float32 or None.
    The plan and workspace are torch CUDA tensors owned by this object.
    """

    def __init__(self, out_f: int, in_f: int, row: torch.Tensor, col: torch.Tensor, val: torch.Tensor,
                 bias: Optional[torch.Tensor] = None, max_batch: int = 1024, validate: bool = False,
                 stream=None):
        if not (row.is_cuda and col.is_cuda and val.is_cuda):
            raise ValueError("row, col and val must be CUDA tensors")
        if row.dtype != torch.int32 or col.dtype != torch.int32:
            raise ValueError("row and col must be int32")
        self.out_f, self.in_f = int(out_f), int(in_f)
        self.row, self.col, self.val = row.contiguous(), col.contiguous(), val.contiguous()
        self.bias = None if bias is None else bias.contiguous().float()
        self.nnz = int(self.row.numel())
        self.max_batch = int(max_batch)
        self.dtype = val.dtype
        code = dtype_code(val.dtype)
        plan_b, ws_b = snack_query_sizes(self.out_f, self.in_f, self.nnz, self.max_batch, code, code)
        dev = val.device
        self.plan = torch.empty(plan_b, dtype=torch.uint8, device=dev)
        self.ws = torch.empty(ws_b, dtype=torch.uint8, device=dev)
        self.handle = snack_create(self.out_f, self.in_f, self.nnz, self.max_batch, code, code, self.row, self.col,
                                   self.plan, self.ws, validate, stream)

    def close(self) -> None:
        if getattr(self, "handle", None):
            snack_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        x = x.contiguous()
        y = out if out is not None else torch.empty((x.shape[0], self.out_f), dtype=self.dtype, device=x.device)
        snack_spmm_fwd(self.handle, self.row, self.col, self.val, x, x.shape[0], self.bias, y, self.ws, stream)
        return y

    def forward_gelu(self, x: torch.Tensor, keep_pre: bool = True, stream=None):
        """GELU(x W^T + b); returns (y, pre) with pre None unless keep_pre."""
        x = x.contiguous()
        y = torch.empty((x.shape[0], self.out_f), dtype=self.dtype, device=x.device)
        pre = torch.empty_like(y) if keep_pre else None
        snack_spmm_fwd_gelu(self.handle, self.row, self.col, self.val, x, x.shape[0], self.bias, pre, y, self.ws,
                            stream)
        return y, pre

    def forward_adapted(self, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, which: torch.Tensor,
                        scales: Optional[torch.Tensor] = None, keep: bool = False, stream=None):
        """x W^T + b with each row's low-rank adapter beside it (see adapt); with keep, (y, h) for adapt_grad."""
        x = x.contiguous()
        y = self.forward(x, stream=stream)
        return adapt(x, y, a, b, which, scales, out=y, keep=keep, stream=stream)

    def grad_input_gelu(self, dy: torch.Tensor, x_pre: torch.Tensor, stream=None) -> torch.Tensor:
        """(dy W) * GELU'(x_pre): the gradient at the pre-activation of this layer's input."""
        dy, x_pre = dy.contiguous(), x_pre.contiguous()
        dx = torch.empty((dy.shape[0], self.in_f), dtype=self.dtype, device=dy.device)
        snack_spmm_dx_gelu(self.handle, self.row, self.col, self.val, dy, dy.shape[0], x_pre, dx, self.ws, stream)
        return dx

    def grad_input(self, dy: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        dy = dy.contiguous()
        dx = out if out is not None else torch.empty((dy.shape[0], self.in_f), dtype=self.dtype, device=dy.device)
        snack_spmm_dx(self.handle, self.row, self.col, self.val, dy, dy.shape[0], dx, self.ws, stream)
        return dx

    def grad_weight(self, x: torch.Tensor, dy: torch.Tensor, want_db: bool = True, stream=None):
        x, dy = x.contiguous(), dy.contiguous()
        dw = torch.empty(self.nnz, dtype=torch.float32, device=x.device)
        db = torch.empty(self.out_f, dtype=torch.float32, device=x.device) if want_db else None
        snack_sddmm_dw(self.handle, self.row, self.col, x, dy, x.shape[0], dw, db, self.ws, stream)
        return dw, db

    def backward(self, x: torch.Tensor, dy: torch.Tensor, want_db: bool = True, stream=None):
        """(dX, dW, db) in one call (fused single pass when the batch fits one tile)."""
        x, dy = x.contiguous(), dy.contiguous()
        dx = torch.empty((dy.shape[0], self.in_f), dtype=self.dtype, device=dy.device)
        dw = torch.empty(self.nnz, dtype=torch.float32, device=x.device)
        db = torch.empty(self.out_f, dtype=torch.float32, device=x.device) if want_db else None
        snack_backward(self.handle, self.row, self.col, self.val, x, dy, x.shape[0], dx, dw, db, self.ws, stream)
        return dx, dw, db

    def restructure(self, n_prune: int, seed: int, step: int, stream=None) -> torch.Tensor:
        """Prune/regrow in place of this layer's pattern; returns src index (-1 = regrown)."""
        need = snack_restructure_workspace_size(self.handle, n_prune)
        ws = self.ws if need <= _nbytes(self.ws) else torch.empty(need, dtype=torch.uint8, device=self.val.device)
        row_o = torch.empty_like(self.row)
        col_o = torch.empty_like(self.col)
        val_o = torch.empty_like(self.val)
        src_o = torch.empty_like(self.row)
        snack_restructure(self.handle, self.row, self.col, self.val, n_prune, seed, step, row_o, col_o, val_o,
                          src_o, ws, stream)
        self.row, self.col, self.val = row_o, col_o, val_o
        return src_o

    def restructure_rows(self, n_per_row: int, seed: int, step: int, stream=None) -> torch.Tensor:
        """Per-row (constant fan-in) prune/regrow in place; returns src index (-1 = regrown)."""
        need = snack_restructure_rows_workspace_size(self.handle, n_per_row)
        ws = self.ws if need <= _nbytes(self.ws) else torch.empty(need, dtype=torch.uint8, device=self.val.device)
        row_o = torch.empty_like(self.row)
        col_o = torch.empty_like(self.col)
        val_o = torch.empty_like(self.val)
        src_o = torch.empty_like(self.row)
        snack_restructure_rows(self.handle, self.row, self.col, self.val, n_per_row, seed, step, row_o, col_o, val_o,
                               src_o, ws, stream)
        self.row, self.col, self.val = row_o, col_o, val_o
        return src_o


class _SparseLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, val, layer: SparseLinear):
        if val.data_ptr() != layer.val.data_ptr():
            raise ValueError("val must be the layer's value tensor")
        ctx.layer = layer
        ctx.save_for_backward(x)
        return layer.forward(x)

    @staticmethod
    def backward(ctx, dy):
        (x,) = ctx.saved_tensors
        layer = ctx.layer
        dy = dy.contiguous().to(layer.dtype)
        dx = layer.grad_input(dy) if ctx.needs_input_grad[0] else None
        dw = layer.grad_weight(x, dy, want_db=False)[0] if ctx.needs_input_grad[1] else None
        if dw is not None and layer.dtype != torch.float32:
            dw = dw.to(layer.dtype)
        return dx, dw, None


def sparse_linear(x: torch.Tensor, layer: SparseLinear) -> torch.Tensor:
    """Autograd-aware Y = X W^T + b; gradients flow to x and to layer.val."""
    return _SparseLinearFn.apply(x, layer.val, layer)


# ------------------------------------------------------------- language-model operators
#
# Plain functions on CUDA tensors (float32 or bfloat16; ids and targets int32 or
# int64).  Outputs and workspaces come from torch's allocator, on the stream
# that the kernels run on: torch's current one, or `stream`.  Tensors that a call
# writes in place count as modified (autograd refuses to use what it saved of them).


class _On:
    """The stream of a call, entered as torch's current one where it is not (and its device with it)."""

    def __init__(self, device: torch.device, stream):
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            # the default stream's handle is 0, of which ExternalStream makes a stream of its own
            stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
        if stream is not None and stream.device != device:
            raise ValueError("the stream belongs to another device than the tensors")
        self.outer = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.outer.__enter__()

    def __exit__(self, *exc):
        self.outer.__exit__(*exc)


def _here(t: torch.Tensor, stream, *others) -> bool:
    """Whether a call on t can run as things stand (torch's current device and stream); all tensors on one GPU."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError("all tensors must be on one CUDA device")
    return stream is None and dev == torch._C._cuda_getDevice()


def _matrix(t: torch.Tensor):
    """t (copied where its rows are not contiguous), its address, rows, width and row step."""
    if t.dim() != 2:
        raise ValueError("expected a matrix")
    rows, width = t.shape
    step, one = t.stride()
    if (one != 1 and width != 1) or step < width:
        t, step = t.contiguous(), width
    return t, t.data_ptr(), rows, width, step


def _code(table, dtype) -> int:
    try:
        return table[dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {dtype}") from None


_DTYPES = {torch.float32: SNACK_F32, torch.bfloat16: SNACK_BF16}
_INDICES = {torch.int32: SNACK_I32, torch.int64: SNACK_I64}


def _out_rows(out: torch.Tensor, rows: int, width: int, dtype) -> torch.Tensor:
    if tuple(out.shape) != (rows, width) or out.dtype != dtype or (width > 1 and out.stride(1) != 1) \
            or (rows > 1 and out.stride(0) < width):
        raise ValueError(f"out must be a {dtype} matrix [{rows}, {width}] with contiguous rows")
    return out


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


# Workspace sizes are functions of the shapes alone (and, for xent, of the rows' alignment).
_embed_grad_ws = functools.lru_cache(maxsize=256)(snack_embed_grad_workspace_size)


@functools.lru_cache(maxsize=256)
def _clip_ws(n: int) -> int:
    return snack_clip_workspace_size([0] * n, [SNACK_F32] * n)


@functools.lru_cache(maxsize=256)
def _xent_ws(device: int, x_bits: int, x_ld: int, n: int, w_bits: int, w_ld: int, vocab: int, width: int, t: int,
             grad: int) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_xent_workspace_size",
           load().snack_xent_workspace_size(x_bits, x_ld, n, w_bits, w_ld, vocab, width, t, grad, ctypes.byref(b)))
    return b.value


def embed(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
          stream=None) -> torch.Tensor:
    """scale * table[ids], zeros for an id outside the table; ids of any shape, the result has that shape plus the width."""
    if not _here(table, stream, ids, out):
        with _On(table.device, stream):
            return embed(ids, table, scale, out)
    tab, addr, vocab, width, ld = _matrix(table)
    flat, kind = ids.contiguous(), tab.dtype
    n = flat.numel()
    y = torch.empty((n, width), dtype=kind, device=tab.device) if out is None else _out_rows(out, n, width, kind)
    st = (_lib or load()).snack_embed_fwd(flat.data_ptr(), _code(_INDICES, flat.dtype), n, addr, ld, vocab, width,
                                          _code(_DTYPES, kind), float(scale), y.data_ptr(), width if out is None else y.stride(0),
                                          _raw_stream(None))
    if st:
        _check("snack_embed_fwd", st)
    if out is not None:
        increment_version(out)
    return y if out is not None or ids.dim() == 1 else y.view(*ids.shape, width)


def embed_grad(ids: torch.Tensor, dout: torch.Tensor, vocab: int, scale: float = 1.0,
               out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """The gradient of embed's table, [vocab, width] in dout's type.  With accumulate the sums are added to `out`."""
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if not _here(dout, stream, ids, out):
        with _On(dout.device, stream):
            return embed_grad(ids, dout, vocab, scale, out, accumulate)
    d, addr, rows, width, ld = _matrix(dout if dout.dim() == 2 else dout.reshape(-1, dout.shape[-1]))
    flat, kind = ids.contiguous(), d.dtype
    n = flat.numel()
    if rows != n:
        raise ValueError("dout needs one row per id")
    g = torch.empty((vocab, width), dtype=kind, device=d.device) if out is None else _out_rows(out, vocab, width, kind)
    nbytes = _embed_grad_ws(n, vocab, width)
    ws = _workspace(nbytes, d.device)
    st = (_lib or load()).snack_embed_grad(flat.data_ptr(), _code(_INDICES, flat.dtype), n, addr, ld, vocab, width,
                                           _code(_DTYPES, kind), float(scale), 1 if accumulate else 0, g.data_ptr(),
                                           width if out is None else g.stride(0), ws.data_ptr(), max(nbytes, 256),
                                           _raw_stream(None))
    if st:
        _check("snack_embed_grad", st)
    if out is not None:
        increment_version(out)
    return g


class _EmbedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return embed(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        return embed_grad(ids, dy, ctx.vocab, ctx.scale), None, None


def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """Autograd-aware embed; the gradient flows to table."""
    return _EmbedFn.apply(table, ids, scale)


def clip_grad_norm(grads, max_norm: float, out=None, stream=None) -> torch.Tensor:
    """The 2-norm over all gradients (a float32 CUDA scalar); scales them so that it is at most max_norm.

    grads: a sequence of contiguous CUDA tensors, float32 and bfloat16 as they
    come.  The clipped gradients go to `out` (tensors of the same types and
    sizes), or in place when it is None.  No output may overlap another tensor
    of the call (a gradient that several parameters share is given once).
    """
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    first = grads[0]
    if not _here(first, stream):
        with _On(first.device, stream):
            return clip_grad_norm(grads, max_norm, out)
    # one call over all tensors per property: a model has hundreds of gradients
    T = torch.Tensor
    numel, dtypes = list(map(T.numel, grads)), [g.dtype for g in grads]
    addr = list(map(T.data_ptr, grads))
    if not all(map(T.is_contiguous, grads)) or set(map(T.get_device, grads)) != {first.get_device()}:
        raise ValueError("gradients must be contiguous tensors on one CUDA device")
    to, outs = addr, grads
    if out is not None:
        outs = list(out)
        if list(map(T.numel, outs)) != numel or [o.dtype for o in outs] != dtypes \
                or not all(map(T.is_contiguous, outs)) or set(map(T.get_device, outs)) != {first.get_device()}:
            raise ValueError("out must hold contiguous tensors of the gradients' types and sizes, on their device")
        to = list(map(T.data_ptr, outs))
    norm = torch.empty((), dtype=torch.float32, device=first.device)
    types = list(map(_DTYPES.get, dtypes))
    if None in types:
        raise ValueError("gradients must be float32 or bfloat16")
    ws = _workspace(_clip_ws(len(grads)), first.device)
    snack_clip_grad_norm(addr, to, numel, types, float(max_norm), norm, ws)
    increment_version(outs)
    return norm


def _xent_args(x, w, targets, reduction, grad):
    """What both calls take of x, w and targets, the reduction, and a workspace; and x, w, targets to keep alive."""
    x, xa, n, width, x_ld = _matrix(x)
    w, wa, vocab, w_width, w_ld = _matrix(w)
    kind = w.dtype
    if width != w_width or x.dtype != kind:
        raise ValueError("x [n, width] and w [vocab, width] must have one type and width")
    if targets.numel() != n:
        raise ValueError("targets needs one entry per row of x")
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}")
    targets = targets.contiguous()
    code = _code(_DTYPES, kind)
    # of the addresses, their place within 256 bytes
    nbytes = max(256, _xent_ws(x.get_device(), xa % 256, x_ld, n, wa % 256, w_ld, vocab, width, code, grad))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    args = (xa, x_ld, n, wa, w_ld, vocab, width, code, targets.data_ptr(), _code(_INDICES, targets.dtype),
            REDUCTIONS[reduction])
    return args, ws, nbytes, (x, w, targets)


def xent(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, reduction: str = "mean", stream=None):
    """Softmax cross entropy of x w^T against targets, without the logits: (loss, state).

    A target outside the vocabulary (such as -100) is not trained on.  state
    (float32, n + 1) is what xent_grad needs beside the same arguments.
    """
    if not _here(x, stream, w, targets):
        with _On(x.device, stream):
            return xent(x, w, targets, reduction)
    args, ws, nbytes, kept = _xent_args(x, w, targets, reduction, 0)
    n, dev = args[2], x.device
    loss = torch.empty((n,) if reduction == "none" else (), dtype=torch.float32, device=dev)
    state = torch.empty(n + 1, dtype=torch.float32, device=dev)
    if n or reduction != "none":
        st = (_lib or load()).snack_xent_fwd(*args, loss.data_ptr(), state.data_ptr(), ws.data_ptr(), nbytes,
                                             _raw_stream(None))
        if st:
            _check("snack_xent_fwd", st)
    return loss, state


def xent_grad(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, state: torch.Tensor,
              dloss: Optional[torch.Tensor] = None, reduction: str = "mean", want_dx: bool = True,
              want_dw: bool = True, stream=None):
    """(dx, dw) of xent for an upstream gradient dloss (1 when None; one value per row for "none")."""
    if not _here(x, stream, w, targets, state, dloss):
        with _On(x.device, stream):
            return xent_grad(x, w, targets, state, dloss, reduction, want_dx, want_dw)
    args, ws, nbytes, kept = _xent_args(x, w, targets, reduction, 1)
    n, width, vocab, kind, dev = args[2], args[6], args[5], x.dtype, x.device
    if state.dtype != torch.float32 or state.numel() != n + 1 or not state.is_contiguous():
        raise ValueError("state must be what xent returned for these arguments")
    if dloss is not None:
        if dloss.numel() != (n if reduction == "none" else 1):
            raise ValueError("dloss has the loss's shape")
        dloss = dloss.contiguous().float()
    elif reduction == "none":
        raise ValueError('reduction "none" needs dloss')
    dx = torch.empty((n, width), dtype=kind, device=dev) if want_dx else None
    dw = torch.empty((vocab, width), dtype=kind, device=dev) if want_dw else None
    st = (_lib or load()).snack_xent_bwd(*args, state.data_ptr(), _addr(dloss), _addr(dx), width, _addr(dw), width,
                                         ws.data_ptr(), nbytes, _raw_stream(None))
    if st:
        _check("snack_xent_bwd", st)
    return dx, dw


class _XentFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, targets, reduction):
        loss, state = xent(x, w, targets, reduction)
        ctx.save_for_backward(x, w, targets, state)
        ctx.reduction = reduction
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x, w, targets, state = ctx.saved_tensors
        dx, dw = xent_grad(x, w, targets, state, dloss, ctx.reduction, ctx.needs_input_grad[0], ctx.needs_input_grad[1])
        return dx, dw, None, None


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, reduction: str = "mean"):
    """Autograd-aware xent: the loss alone; gradients flow to x and w."""
    return _XentFn.apply(x, w, targets, reduction)


@functools.lru_cache(maxsize=256)
def _score_ws(device: int, x_bits: int, x_ld: int, n: int, w_bits: int, w_ld: int, vocab: int, width: int, t: int, top: int,
              grad: int) -> int:
    b = ctypes.c_size_t(0)
    _check("snack_score_workspace_size",
           load().snack_score_workspace_size(x_bits, x_ld, n, w_bits, w_ld, vocab, width, t, top, grad, ctypes.byref(b)))
    return b.value


def _score_args(x, w, targets, top, grad):
    """What both calls take of x, w and targets, and a workspace; and what to keep alive."""
    x, xa, n, width, x_ld = _matrix(x)
    w, wa, vocab, w_width, w_ld = _matrix(w)
    kind = w.dtype
    if width != w_width or x.dtype != kind:
        raise ValueError("x [n, width] and w [vocab, width] must have one type and width")
    ids, ids_t = None, SNACK_I64
    if targets is not None:
        if targets.numel() != n:
            raise ValueError("targets needs one entry per row of x")
        targets = targets.contiguous()
        ids, ids_t = targets.data_ptr(), _code(_INDICES, targets.dtype)
    code = _code(_DTYPES, kind)
    nbytes = max(256, _score_ws(x.get_device(), xa % 256, x_ld, n, wa % 256, w_ld, vocab, width, code, top, grad))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    return (xa, x_ld, n, wa, w_ld, vocab, width, code, ids, ids_t), ws, nbytes, (x, w, targets)


def score(x: torch.Tensor, w: torch.Tensor, targets: Optional[torch.Tensor] = None, top: int = 0, stream=None):
    """Log probabilities of targets under softmax(x w^T), entropies, likeliest tokens: (logp, entropy, ids, top_logp, state).

    logp is None without targets; ids (int64, [n, top], likeliest first, of equal
    logits the lower id) and top_logp are None where top is 0.  A row whose target is
    outside the vocabulary (such as -100) is not scored: its results are 0, its ids
    -1.  state (float32, [2, n]) is what score_grad needs beside the same arguments.
    """
    if not _here(x, stream, w, targets):
        with _On(x.device, stream):
            return score(x, w, targets, top)
    top = int(top)
    args, ws, nbytes, kept = _score_args(x, w, targets, top, 0)
    n, dev = args[2], x.device
    logp = torch.empty(n, dtype=torch.float32, device=dev) if targets is not None else None
    entropy = torch.empty(n, dtype=torch.float32, device=dev)
    ids = torch.empty((n, top), dtype=torch.int64, device=dev) if top else None
    top_logp = torch.empty((n, top), dtype=torch.float32, device=dev) if top else None
    state = torch.empty((2, n), dtype=torch.float32, device=dev)
    st = (_lib or load()).snack_score_fwd(*args, _addr(logp), entropy.data_ptr(), top, _addr(ids), _addr(top_logp),
                                          state.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(None))
    if st:
        _check("snack_score_fwd", st)
    return logp, entropy, ids, top_logp, state


def score_grad(x: torch.Tensor, w: torch.Tensor, targets: Optional[torch.Tensor], state: torch.Tensor,
               dlogp: Optional[torch.Tensor] = None, dentropy: Optional[torch.Tensor] = None, want_dx: bool = True,
               want_dw: bool = True, stream=None):
    """(dx, dw) of score for upstream gradients of its log probabilities and entropies (None: 0)."""
    if not _here(x, stream, w, targets, state, dlogp, dentropy):
        with _On(x.device, stream):
            return score_grad(x, w, targets, state, dlogp, dentropy, want_dx, want_dw)
    args, ws, nbytes, kept = _score_args(x, w, targets, 0, 1)
    n, vocab, width, kind, dev = args[2], args[5], args[6], x.dtype, x.device
    if state.dtype != torch.float32 or tuple(state.shape) != (2, n) or not state.is_contiguous():
        raise ValueError("state must be what score returned for these arguments")
    if targets is None and dlogp is not None:
        raise ValueError("dlogp needs targets")
    up = []
    for d in (dlogp, dentropy):
        if d is not None and d.numel() != n:
            raise ValueError("dlogp and dentropy need one entry per row of x")
        up.append(None if d is None else d.contiguous().float())
    dx = torch.empty((n, width), dtype=kind, device=dev) if want_dx else None
    dw = torch.empty((vocab, width), dtype=kind, device=dev) if want_dw else None
    st = (_lib or load()).snack_score_bwd(*args, state.data_ptr(), _addr(up[0]), _addr(up[1]), _addr(dx), width, _addr(dw),
                                          width, ws.data_ptr(), nbytes, _raw_stream(None))
    if st:
        _check("snack_score_bwd", st)
    return dx, dw


class _ScoreFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, targets):
        logp, entropy, _, _, state = score(x, w, targets)
        ctx.save_for_backward(x, w, targets, state)
        return logp, entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy):
        x, w, targets, state = ctx.saved_tensors
        dx, dw = score_grad(x, w, targets, state, dlogp, dentropy, ctx.needs_input_grad[0], ctx.needs_input_grad[1])
        return dx, dw, None


def token_logprobs(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor):
    """Autograd-aware score: (log probabilities of targets, entropies); gradients flow to x and w."""
    return _ScoreFn.apply(x, w, targets)


_adapt_ws = functools.lru_cache(maxsize=256)(snack_adapt_workspace_size)


def _adapt_args(x, a, b, which, scales):
    """What both calls take of x and the adapters, and a workspace; and what to keep alive."""
    x, xa, n, width, x_ld = _matrix(x)
    kind, shape_a, shape_b = x.dtype, a.shape, b.shape
    if len(shape_a) != 3 or len(shape_b) != 3:
        raise ValueError("a must be [adapters, rank, width of x] and b [adapters, width of the output, rank]")
    adapters, rank, in_f = shape_a
    if shape_b[0] != adapters or shape_b[2] != rank or in_f != width:
        raise ValueError("a must be [adapters, rank, width of x] and b [adapters, width of the output, rank]")
    if a.dtype != kind or b.dtype != kind:
        raise ValueError("x, a and b must have one type")
    if which.numel() != n:
        raise ValueError("which needs one entry per row of x")
    scales_addr = None
    if scales is not None:
        if scales.dtype != torch.float32 or scales.numel() != adapters:
            raise ValueError("scales must hold one float32 value per adapter")
        scales = scales.contiguous()
        scales_addr = scales.data_ptr()
    a, b, which = a.contiguous(), b.contiguous(), which.contiguous()
    nbytes = _adapt_ws(n, adapters, rank) or 256
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    args = (xa, x_ld, n, a.data_ptr(), b.data_ptr(), adapters, rank, width, shape_b[1], _code(_DTYPES, kind), which.data_ptr(),
            _code(_INDICES, which.dtype), scales_addr)
    return args, ws, nbytes, (x, a, b, which, scales)


def adapt(x: torch.Tensor, base: Optional[torch.Tensor], a: torch.Tensor, b: torch.Tensor, which: torch.Tensor,
          scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, keep: bool = False, stream=None):
    """base + scales[k] * (x A_k^T) B_k^T, where k = which[i] is the adapter of row i's request.

    x [n, in], base [n, out] (None: 0), a [adapters, rank, in] and b [adapters,
    out, rank] in one type; a row whose entry of which is outside the adapters keeps
    its base.  The result goes to `out`, which may be base.  With keep, returns (y,
    h): h (float32, [n, rank]) is what adapt_grad needs.
    """
    if not _here(x, stream, base, a, b, which, scales, out):
        with _On(x.device, stream):
            return adapt(x, base, a, b, which, scales, out, keep)
    args, ws, nbytes, kept = _adapt_args(x, a, b, which, scales)
    n, rank, out_f, kind = args[2], args[6], args[8], kept[0].dtype
    base_addr, base_ld = None, 0
    if base is not None:
        if base.dtype != kind or base.shape != (n, out_f):
            raise ValueError(f"base must be a {kind} matrix [{n}, {out_f}]")
        if out is not base:
            base, base_addr, _, _, base_ld = _matrix(base)
    y = torch.empty((n, out_f), dtype=kind, device=x.device) if out is None else _out_rows(out, n, out_f, kind)
    y_ld = out_f if out is None or n < 2 else y.stride(0)
    if base is not None and out is base:
        base_addr, base_ld = y.data_ptr(), y_ld
    h = torch.empty((n, rank), dtype=torch.float32, device=x.device) if keep else None
    st = (_lib or load()).snack_adapt_fwd(*args, base_addr, base_ld, y.data_ptr(), y_ld, _addr(h), ws.data_ptr(), nbytes,
                                          _raw_stream(None))
    if st:
        _check("snack_adapt_fwd", st)
    if out is not None:
        increment_version(out)
    return (y, h) if keep else y


def adapt_grad(x: torch.Tensor, dy: torch.Tensor, a: torch.Tensor, b: torch.Tensor, which: torch.Tensor,
               h: Optional[torch.Tensor], scales: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
               want_dx: bool = True, want_da: bool = True, want_db: bool = True, stream=None):
    """(dx, da, db) of adapt for the upstream gradient dy; base's gradient is dy itself.

    dx is the adapters' part alone; given as an argument, it is added to what is
    there (the projection's own input gradient).  h is what adapt kept (needed for db).
    """
    if not _here(x, stream, dy, a, b, which, h, scales, dx):
        with _On(x.device, stream):
            return adapt_grad(x, dy, a, b, which, h, scales, dx, want_dx, want_da, want_db)
    args, ws, nbytes, kept = _adapt_args(x, a, b, which, scales)
    n, adapters, rank, width, out_f, kind = args[2], args[5], args[6], args[7], args[8], kept[0].dtype
    if dy.dtype != kind or dy.shape != (n, out_f):
        raise ValueError(f"dy must be a {kind} matrix [{n}, {out_f}]")
    dy, dy_addr, _, _, dy_ld = _matrix(dy)
    if h is None:
        if want_db:
            raise ValueError("the gradient of b needs h")
    elif h.dtype != torch.float32 or h.shape != (n, rank) or not h.is_contiguous():
        raise ValueError("h must be what adapt kept for these arguments")
    add = dx is not None
    if add:
        _out_rows(dx, n, width, kind)
    elif want_dx:
        dx = torch.empty((n, width), dtype=kind, device=x.device)
    da = torch.empty_like(kept[1]) if want_da else None
    db = torch.empty_like(kept[2]) if want_db else None
    dx_ld = 0 if dx is None else width if n < 2 else dx.stride(0)
    st = (_lib or load()).snack_adapt_bwd(*args, _addr(h), dy_addr, dy_ld, 1 if add else 0, _addr(dx), dx_ld, _addr(da),
                                          _addr(db), ws.data_ptr(), nbytes, _raw_stream(None))
    if st:
        _check("snack_adapt_bwd", st)
    if add:
        increment_version(dx)
    return dx, da, db


class _AdaptFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, base, a, b, which, scales):
        y, h = adapt(x, base, a, b, which, scales, keep=True)
        ctx.save_for_backward(x, a, b, which, h, scales)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, a, b, which, h, scales = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, da, db = adapt_grad(x, dy, a, b, which, h, scales, None, need[0], need[2], need[3])
        return dx, dy if need[1] else None, da, db, None, None


def adapted(x: torch.Tensor, base: torch.Tensor, a: torch.Tensor, b: torch.Tensor, which: torch.Tensor,
            scales: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Autograd-aware adapt; gradients flow to x, base, a and b.  scales that want one are refused: they get none."""
    if scales is not None and scales.requires_grad and torch.is_grad_enabled():
        raise ValueError("adapted gives scales no gradient: detach them")
    return _AdaptFn.apply(x, base, a, b, which, scales)
