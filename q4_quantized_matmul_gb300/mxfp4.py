"""MXFP4 weights, their products, and the experts' side of a mixture of experts.

Bindings of the same names in include/q4q.h, which states the formats and formulas.
Matrices are torch CUDA tensors (float32, float16 or bfloat16, contiguous), MXFP4
matrices uint8 tensors of q4q_mxfp4_size bytes; outputs, workspaces and the stream
default to new tensors and the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import Q4QError, _lib

Q4Q_ACTS_MXFP4 = 0
Q4Q_ACTS_MXFP8 = 1

_TYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


# These calls take a few microseconds on the GPU, so what surrounds them is kept short: the
# C functions are looked up once, pointers are plain integers, and the device is switched
# only where the tensors lie on another one than the current.

_current_device = torch.cuda.current_device
_current_stream = torch._C._cuda_getCurrentRawStream


class _Lib:
    """The loaded library's functions, each looked up at its first use."""

    def __getattr__(self, name):
        fn = getattr(_lib.load(), name)
        setattr(self, name, fn)
        return fn


_c = _Lib()


def _on_device_of(fn):
    """Run with the device of the first argument current."""
    @functools.wraps(fn)
    def wrapper(t, *args, **kwargs):
        if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != _current_device():
            with torch.cuda.device(t.device):
                return fn(t, *args, **kwargs)
        return fn(t, *args, **kwargs)
    return wrapper


def _check(fn: str, status: int):
    if status:
        raise Q4QError(fn, status)


def _stream(stream, like: torch.Tensor) -> int:
    """The cudaStream_t of a torch stream or integer; the current stream of `like`'s device for None."""
    if stream is None:
        return _current_stream(like.get_device())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _type(t: torch.Tensor, name: str) -> int:
    type_ = _TYPE.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if type_ is None:
        raise TypeError("%s must be a float32, float16 or bfloat16 tensor" % name)
    return type_


def _ptr(t: torch.Tensor, name: str, dtype: Optional[torch.dtype], count: int) -> int:
    """The address of a contiguous CUDA tensor of `dtype` (any for None) that holds `count` elements (bytes for None)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be a %s tensor" % (name, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    have = t.numel() if dtype is not None else t.numel() * t.element_size()
    if have < count:
        raise ValueError("%s holds %d %s, the call reads or writes %d" % (
            name, have, "elements" if dtype is not None else "bytes", count))
    return t.data_ptr()


def _new(like: torch.Tensor, shape, dtype: torch.dtype, stream) -> torch.Tensor:
    """A tensor of the call's own, whose memory the allocator keeps from other users until `stream` is past the call."""
    t = torch.empty(shape, dtype=dtype, device=like.device)
    if stream is not None:
        t.record_stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream))
    return t


def _scratch(like: torch.Tensor, size: int, stream) -> Optional[torch.Tensor]:
    return _new(like, (size,), torch.uint8, stream) if size else None


def _bytes(workspace: Optional[torch.Tensor]):
    """Address and size of a workspace."""
    if workspace is None:
        return None, 0
    return _ptr(workspace, "workspace", None, 0), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=4096)
def q4q_mxfp4_size(ne00: int, ne01: int) -> int:
    """Bytes of one MXFP4 matrix."""
    n = ctypes.c_size_t(0)
    _check("q4q_mxfp4_size", _c.q4q_mxfp4_size(ne00, ne01, ctypes.byref(n)))
    return int(n.value)


@_on_device_of
def q4q_quantize_mxfp4(src: torch.Tensor, dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """[rows, K] -> uint8 [q4q_mxfp4_size(K, rows)]; [matrices, rows, K] -> one row of bytes for each."""
    type_ = _type(src, "src")
    if src.dim() not in (2, 3):
        raise ValueError("src must be [rows, K] or [matrices, rows, K]")
    nmats, (nrows, ncols) = (src.shape[0] if src.dim() == 3 else 1), src.shape[-2:]
    size = q4q_mxfp4_size(ncols, nrows)
    if dst is None:
        dst = _new(src, (nmats, size) if src.dim() == 3 else (size,), torch.uint8, stream)
    _check("q4q_quantize_mxfp4", _c.q4q_quantize_mxfp4(
        _ptr(src, "src", src.dtype, 0), type_, _ptr(dst, "dst", None, nmats * size), ncols, nrows, nmats, _stream(stream, src)))
    return dst


@_on_device_of
def q4q_get_rows_mxfp4(src0: torch.Tensor, ne00: int, ne01: int, ids: Optional[torch.Tensor] = None,
                       n_ids: Optional[int] = None, dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows ids of an MXFP4 matrix [ne00, ne01] as fp32 [n_ids, ne00]; ids None = rows 0..n_ids-1."""
    if ids is not None:
        n_ids = ids.numel()
    elif n_ids is None:
        n_ids = ne01
    if dst is None:
        dst = _new(src0, (n_ids, ne00), torch.float32, stream)
    if n_ids == 0:
        return dst
    _check("q4q_get_rows_mxfp4", _c.q4q_get_rows_mxfp4(
        _ptr(src0, "src0", None, q4q_mxfp4_size(ne00, ne01)), ne00, ne01,
        _ptr(ids, "ids", torch.int32, n_ids) if ids is not None else None, n_ids,
        _ptr(dst, "dst", torch.float32, n_ids * ne00), _stream(stream, src0)))
    return dst


def _acts(src1: torch.Tensor) -> torch.Tensor:
    return src1 if src1.dim() == 2 else src1.reshape(-1, src1.shape[-1])


def _out(dst: Optional[torch.Tensor], dtype: Optional[torch.dtype], like: torch.Tensor, rows: int, cols: int, stream) -> torch.Tensor:
    if dst is not None:
        return dst
    return _new(like, (rows, cols), like.dtype if dtype is None else dtype, stream)


@functools.lru_cache(maxsize=4096)
def _dense_workspace(ne00: int, ne01: int, ne11: int, acts: int, device: int) -> int:
    n = ctypes.c_size_t(0)
    _check("q4q_mul_mat_mxfp4_workspace_size",
           _c.q4q_mul_mat_mxfp4_workspace_size(ne00, ne01, ne11, acts, ctypes.byref(n)))
    return int(n.value)


def q4q_mul_mat_mxfp4_workspace_size(ne00: int, ne01: int, ne11: int, acts: int = Q4Q_ACTS_MXFP8) -> int:
    """Bytes of workspace of q4q_mul_mat_mxfp4 on the current device."""
    return _dense_workspace(ne00, ne01, ne11, int(acts), _current_device())


@_on_device_of
def q4q_mul_mat_mxfp4(src0: torch.Tensor, ne00: int, ne01: int, src1: torch.Tensor, acts: int = Q4Q_ACTS_MXFP8,
                      dst: Optional[torch.Tensor] = None, dst_dtype: Optional[torch.dtype] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None, flags: int = 0) -> torch.Tensor:
    """src1 [ne11, ne00] times the MXFP4 matrix src0 [ne00, ne01], -> [ne11, ne01] of dst_dtype (src1's by default)."""
    type_ = _type(src1, "src1")
    x = _acts(src1)
    ne11, ne10 = x.shape
    dst = _out(dst, dst_dtype, x, ne11, ne01, stream)
    if ne01 * ne11 == 0:
        return dst
    if workspace is None:
        workspace = _scratch(x, _dense_workspace(ne00, ne01, ne11, acts, _current_device()), stream)
    _check("q4q_mul_mat_mxfp4", _c.q4q_mul_mat_mxfp4(
        _ptr(src0, "src0", None, q4q_mxfp4_size(ne00, ne01)), ne00, ne01, _ptr(x, "src1", src1.dtype, 0), type_, ne10, ne11,
        acts, _ptr(dst, "dst", dst.dtype, ne11 * ne01), _type(dst, "dst"), *_bytes(workspace), flags, _stream(stream, x)))
    return dst


@_on_device_of
def q4q_debug_mul_mat_mxfp4_timeout(src0: torch.Tensor, ne00: int, ne01: int, src1: torch.Tensor, acts: int,
                                    limit_ns: int, stream=None) -> torch.Tensor:
    """q4q_mul_mat_mxfp4 with its first CTA's first stage left out and every wait bounded by limit_ns:
    q4q_device_status() then reports Q4Q_ERR_TIMEOUT (6) and the result is incomplete."""
    x = _acts(src1)
    dst = _new(x, (x.shape[0], ne01), torch.float32, stream)
    workspace = _new(x, q4q_mul_mat_mxfp4_workspace_size(ne00, ne01, x.shape[0], acts), torch.uint8, stream)
    _check("q4q_debug_mul_mat_mxfp4_timeout", _c.q4q_debug_mul_mat_mxfp4_timeout(
        _ptr(src0, "src0", None, q4q_mxfp4_size(ne00, ne01)), ne00, ne01, _ptr(x, "src1", torch.float32, x.shape[0] * ne00),
        x.shape[0], acts, dst.data_ptr(), workspace.data_ptr(), workspace.numel(), limit_ns, _stream(stream, x)))
    return dst


# ------------------------------------------------------------------ experts --

@_on_device_of
def q4q_moe_sort(ids: torch.Tensor, n_experts: int, first: Optional[torch.Tensor] = None, slot: Optional[torch.Tensor] = None,
                 row: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Sort the choices ids int32 [tokens, top_k] by expert: (first [n_experts + 1], slot, row [tokens * top_k])."""
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    n_tokens, top_k = ids.shape
    n = n_tokens * top_k
    if first is None:
        first = _new(ids, (n_experts + 1,), torch.int32, stream)
    if slot is None:
        slot = _new(ids, (n,), torch.int32, stream)
    if row is None:
        row = _new(ids, (n,), torch.int32, stream)
    _check("q4q_moe_sort", _c.q4q_moe_sort(
        _ptr(ids, "ids", torch.int32, n), n_tokens, top_k, n_experts, _ptr(first, "first", torch.int32, n_experts + 1),
        _ptr(slot, "slot", torch.int32, n), _ptr(row, "row", torch.int32, n), _stream(stream, ids)))
    return first, slot, row


def _row_args(first: torch.Tensor, row: torch.Tensor, n: int):
    return _ptr(first, "first", torch.int32, 1), first.numel() - 1, _ptr(row, "row", torch.int32, n)


@_on_device_of
def q4q_moe_gather(src: torch.Tensor, first: torch.Tensor, row: torch.Tensor, top_k: int, dst: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Tokens [tokens, ne0] to their experts' rows [tokens * top_k, ne0]."""
    type_, (n, ne0) = _type(src, "src"), src.shape
    dst = _out(dst, None, src, n * top_k, ne0, stream)
    f, e, r = _row_args(first, row, n * top_k)
    _check("q4q_moe_gather", _c.q4q_moe_gather(
        _ptr(src, "src", src.dtype, 0), type_, ne0, n, top_k, f, e, r, _ptr(dst, "dst", src.dtype, n * top_k * ne0),
        _stream(stream, src)))
    return dst


@_on_device_of
def q4q_moe_gather_back(d_dst: torch.Tensor, first: torch.Tensor, row: torch.Tensor, top_k: int,
                        d_src: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of q4q_moe_gather: sorted rows [tokens * top_k, ne0] summed to their tokens [tokens, ne0]."""
    type_, (slots, ne0) = _type(d_dst, "d_dst"), d_dst.shape
    if top_k < 1 or slots % top_k:
        raise ValueError("d_dst must hold top_k rows for each token")
    n = slots // top_k
    d_src = _out(d_src, None, d_dst, n, ne0, stream)
    f, e, r = _row_args(first, row, slots)
    _check("q4q_moe_gather_back", _c.q4q_moe_gather_back(
        _ptr(d_dst, "d_dst", d_dst.dtype, 0), type_, ne0, n, top_k, f, e, r, _ptr(d_src, "d_src", d_dst.dtype, n * ne0),
        _stream(stream, d_dst)))
    return d_src


@_on_device_of
def q4q_moe_combine(rows: torch.Tensor, first: torch.Tensor, row: torch.Tensor, weights: torch.Tensor,
                    dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Experts' rows [tokens * top_k, ne0] weighted (fp32 [tokens, top_k]) and summed to their tokens [tokens, ne0]."""
    type_, (n, top_k), ne0 = _type(rows, "rows"), weights.shape, rows.shape[-1]
    dst = _out(dst, None, rows, n, ne0, stream)
    f, e, r = _row_args(first, row, n * top_k)
    _check("q4q_moe_combine", _c.q4q_moe_combine(
        _ptr(rows, "rows", rows.dtype, n * top_k * ne0), type_, ne0, n, top_k, f, e, r,
        _ptr(weights, "weights", torch.float32, n * top_k), _ptr(dst, "dst", rows.dtype, n * ne0), _stream(stream, rows)))
    return dst


@_on_device_of
def q4q_moe_combine_back(d_dst: torch.Tensor, rows: torch.Tensor, first: torch.Tensor, row: torch.Tensor,
                         weights: torch.Tensor, d_rows: Optional[torch.Tensor] = None,
                         d_weights: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradients of q4q_moe_combine: (d_rows like rows, d_weights fp32 [tokens, top_k])."""
    type_, (n, top_k), ne0 = _type(d_dst, "d_dst"), weights.shape, rows.shape[-1]
    d_rows = _out(d_rows, None, rows, n * top_k, ne0, stream)
    if d_weights is None:
        d_weights = _new(rows, (n, top_k), torch.float32, stream)
    f, e, r = _row_args(first, row, n * top_k)
    _check("q4q_moe_combine_back", _c.q4q_moe_combine_back(
        _ptr(d_dst, "d_dst", rows.dtype, n * ne0), _ptr(rows, "rows", rows.dtype, n * top_k * ne0), type_, ne0, n, top_k, f, e, r,
        _ptr(weights, "weights", torch.float32, n * top_k), _ptr(d_rows, "d_rows", rows.dtype, n * top_k * ne0),
        _ptr(d_weights, "d_weights", torch.float32, n * top_k), _stream(stream, rows)))
    return d_rows, d_weights


@functools.lru_cache(maxsize=4096)
def _id_workspace(ne00: int, ne01: int, n_src1: int, n_rows: int, n_experts: int, acts: int, device: int) -> int:
    n = ctypes.c_size_t(0)
    _check("q4q_mul_mat_id_mxfp4_workspace_size", _c.q4q_mul_mat_id_mxfp4_workspace_size(
        ne00, ne01, n_src1, n_rows, n_experts, acts, ctypes.byref(n)))
    return int(n.value)


def q4q_mul_mat_id_mxfp4_workspace_size(ne00: int, ne01: int, n_src1: int, n_rows: int, n_experts: int,
                                        acts: int = Q4Q_ACTS_MXFP8) -> int:
    """Bytes of workspace of q4q_mul_mat_id_mxfp4 on the current device."""
    return _id_workspace(ne00, ne01, n_src1, n_rows, n_experts, int(acts), _current_device())


@_on_device_of
def q4q_mul_mat_id_mxfp4(src0: torch.Tensor, ne00: int, ne01: int, src1: torch.Tensor, first: torch.Tensor,
                         slot: Optional[torch.Tensor] = None, top_k: int = 1, acts: int = Q4Q_ACTS_MXFP8,
                         dst: Optional[torch.Tensor] = None, dst_dtype: Optional[torch.dtype] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None, flags: int = 0) -> torch.Tensor:
    """The experts' products of the sorted rows, [rows, ne01] of dst_dtype (src1's by default).

    src0: n_experts MXFP4 matrices [ne00, ne01]; first, slot: from q4q_moe_sort.  With slot,
    src1 holds tokens [tokens, ne00] and sorted row r takes token slot[r] // top_k; without,
    src1 holds the sorted rows themselves."""
    type_ = _type(src1, "src1")
    x = _acts(src1)
    n_src1, ne10 = x.shape
    n_experts, n_rows = first.numel() - 1, slot.numel() if slot is not None else n_src1
    dst = _out(dst, dst_dtype, x, n_rows, ne01, stream)
    if ne01 * n_rows == 0:
        return dst
    if workspace is None:
        workspace = _scratch(x, _id_workspace(ne00, ne01, n_src1, n_rows, n_experts, acts, _current_device()), stream)
    _check("q4q_mul_mat_id_mxfp4", _c.q4q_mul_mat_id_mxfp4(
        _ptr(src0, "src0", None, n_experts * q4q_mxfp4_size(ne00, ne01)), ne00, ne01, n_experts, _ptr(x, "src1", src1.dtype, 0),
        type_, ne10, n_src1, _ptr(first, "first", torch.int32, n_experts + 1),
        _ptr(slot, "slot", torch.int32, n_rows) if slot is not None else None, n_rows, top_k, acts,
        _ptr(dst, "dst", dst.dtype, n_rows * ne01), _type(dst, "dst"), *_bytes(workspace), flags, _stream(stream, x)))
    return dst
