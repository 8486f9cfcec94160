"""MXFP4 weights, their products, and the experts' side of a mixture of experts.

Bindings of the same names in include/q4q.h, which states the formats and formulas.
Matrices are torch CUDA tensors (float32, float16 or bfloat16, contiguous), MXFP4
matrices uint8 tensors of q4q_mxfp4_size bytes; outputs, workspaces and the stream
default to new tensors and the current stream of the tensors' device.  Autograd does not
see these calls: their results need no gradient, whatever their inputs need.  The gradients
of gather and combine are calls of their own; the products have none.  The calls
themselves are csrc/q4q_torch.cpp: checks and allocations in C++, because they would
take longer than the kernels in Python.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
from typing import Optional, Tuple

import torch

from . import Q4QError, _dev, _lib

Q4Q_ACTS_MXFP4 = 0
Q4Q_ACTS_MXFP8 = 1

_EXT_PATH = os.path.join(os.path.dirname(_lib.LIB_PATH), "_q4q_torch.so")


class _Ext:
    """The functions of _q4q_torch.so, loaded at the first use.  There is no fallback."""

    def __getattr__(self, name):
        if not os.path.exists(_EXT_PATH):
            raise RuntimeError("_q4q_torch.so is not built (%s); run __graft_entry__.build() first" % _EXT_PATH)
        spec = importlib.util.spec_from_file_location("_q4q_torch", _EXT_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.set_error(Q4QError)
        self.__dict__.update({k: v for k, v in vars(module).items() if not k.startswith("_")})
        return self.__dict__[name]


_ext = _Ext()


def _check(fn: str, status: int):
    if status:
        raise Q4QError(fn, status)


@functools.lru_cache(maxsize=4096)
def q4q_mxfp4_size(ne00: int, ne01: int) -> int:
    """Bytes of one MXFP4 matrix."""
    n = ctypes.c_size_t(0)
    _check("q4q_mxfp4_size", _lib.load().q4q_mxfp4_size(ne00, ne01, ctypes.byref(n)))
    return int(n.value)


def q4q_quantize_mxfp4(src: torch.Tensor, dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """[rows, K] -> uint8 [q4q_mxfp4_size(K, rows)]; [matrices, rows, K] -> one row of bytes for each."""
    return _ext.quantize_mxfp4(src, dst, stream)


def q4q_get_rows_mxfp4(src0: torch.Tensor, ne00: int, ne01: int, ids: Optional[torch.Tensor] = None,
                       n_ids: Optional[int] = None, dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows ids of an MXFP4 matrix [ne00, ne01] as fp32 [n_ids, ne00]; ids None = rows 0..n_ids-1."""
    return _ext.get_rows_mxfp4(src0, ne00, ne01, ids, n_ids, dst, stream)


def q4q_mul_mat_mxfp4_workspace_size(ne00: int, ne01: int, ne11: int, acts: int = Q4Q_ACTS_MXFP8) -> int:
    """Bytes of workspace of q4q_mul_mat_mxfp4 on the current device."""
    n = ctypes.c_size_t(0)
    _check("q4q_mul_mat_mxfp4_workspace_size",
           _lib.load().q4q_mul_mat_mxfp4_workspace_size(ne00, ne01, ne11, int(acts), ctypes.byref(n)))
    return int(n.value)


def q4q_mul_mat_mxfp4(src0: torch.Tensor, ne00: int, ne01: int, src1: torch.Tensor, acts: int = Q4Q_ACTS_MXFP8,
                      dst: Optional[torch.Tensor] = None, dst_dtype: Optional[torch.dtype] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None, flags: int = 0) -> torch.Tensor:
    """src1 [ne11, ne00] times the MXFP4 matrix src0 [ne00, ne01], -> [ne11, ne01] of dst_dtype (src1's by default)."""
    return _ext.mul_mat_mxfp4(src0, ne00, ne01, src1, acts, dst, dst_dtype, workspace, stream, flags)


def q4q_debug_mul_mat_mxfp4_timeout(src0: torch.Tensor, ne00: int, ne01: int, src1: torch.Tensor, acts: int,
                                    limit_ns: int) -> torch.Tensor:
    """q4q_mul_mat_mxfp4 on the current stream with its first CTA's first stage left out and every wait bounded
    by limit_ns: q4q_device_status() then reports Q4Q_ERR_TIMEOUT (6) and the result is incomplete."""
    w = _dev(src0, "src0", q4q_mxfp4_size(ne00, ne01))
    ne11 = src1.shape[0]
    if src1.dtype != torch.float32 or not src1.is_cuda or not src1.is_contiguous() or src1.shape != (ne11, ne00):
        raise TypeError("src1 must be a contiguous float32 CUDA tensor [ne11, ne00]")
    if src1.device != src0.device:
        raise ValueError("src1 is on another device")
    with torch.cuda.device(src1.device):
        dst = torch.empty((ne11, ne01), dtype=torch.float32, device=src1.device)
        workspace = torch.empty(q4q_mul_mat_mxfp4_workspace_size(ne00, ne01, ne11, acts), dtype=torch.uint8, device=src1.device)
        _check("q4q_debug_mul_mat_mxfp4_timeout", _lib.load().q4q_debug_mul_mat_mxfp4_timeout(
            w, ne00, ne01, src1.data_ptr(), ne11, int(acts), dst.data_ptr(), workspace.data_ptr(),
            workspace.numel(), int(limit_ns), torch.cuda.current_stream().cuda_stream))
    return dst


# ------------------------------------------------------------------ experts --

def q4q_moe_sort(ids: torch.Tensor, n_experts: int, first: Optional[torch.Tensor] = None, slot: Optional[torch.Tensor] = None,
                 row: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Sort the choices ids int32 [tokens, top_k] by expert: (first [n_experts + 1], slot, row [tokens * top_k]),
    in one storage where none of them is given."""
    return _ext.moe_sort(ids, n_experts, first, slot, row, stream)


def q4q_moe_gather(src: torch.Tensor, first: torch.Tensor, row: torch.Tensor, top_k: int, dst: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Tokens [tokens, ne0] to their experts' rows [tokens * top_k, ne0]."""
    return _ext.moe_gather(src, first, row, top_k, dst, stream)


def q4q_moe_gather_back(d_dst: torch.Tensor, first: torch.Tensor, row: torch.Tensor, top_k: int,
                        d_src: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of q4q_moe_gather: sorted rows [tokens * top_k, ne0] summed to their tokens [tokens, ne0]."""
    return _ext.moe_gather_back(d_dst, first, row, top_k, d_src, stream)


def q4q_moe_combine(rows: torch.Tensor, first: torch.Tensor, row: torch.Tensor, weights: torch.Tensor,
                    dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Experts' rows [tokens * top_k, ne0] weighted (fp32 [tokens, top_k]) and summed to their tokens [tokens, ne0]."""
    return _ext.moe_combine(rows, first, row, weights, dst, stream)


def q4q_moe_combine_back(d_dst: torch.Tensor, rows: torch.Tensor, first: torch.Tensor, row: torch.Tensor,
                         weights: torch.Tensor, d_rows: Optional[torch.Tensor] = None,
                         d_weights: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradients of q4q_moe_combine: (d_rows like rows, d_weights fp32 [tokens, top_k])."""
    return _ext.moe_combine_back(d_dst, rows, first, row, weights, d_rows, d_weights, stream)


def q4q_mul_mat_id_mxfp4_workspace_size(ne00: int, ne01: int, n_src1: int, n_rows: int, n_experts: int,
                                        acts: int = Q4Q_ACTS_MXFP8) -> int:
    """Bytes of workspace of q4q_mul_mat_id_mxfp4 on the current device."""
    n = ctypes.c_size_t(0)
    _check("q4q_mul_mat_id_mxfp4_workspace_size", _lib.load().q4q_mul_mat_id_mxfp4_workspace_size(
        ne00, ne01, n_src1, n_rows, n_experts, int(acts), ctypes.byref(n)))
    return int(n.value)


def q4q_mul_mat_id_mxfp4(src0: torch.Tensor, ne00: int, ne01: int, src1: torch.Tensor, first: torch.Tensor,
                         slot: Optional[torch.Tensor] = None, top_k: int = 1, acts: int = Q4Q_ACTS_MXFP8,
                         dst: Optional[torch.Tensor] = None, dst_dtype: Optional[torch.dtype] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None, flags: int = 0) -> torch.Tensor:
    """The experts' products of the sorted rows, [rows, ne01] of dst_dtype (src1's by default).

    src0: n_experts MXFP4 matrices [ne00, ne01]; first, slot: from q4q_moe_sort.  With slot,
    src1 holds tokens [tokens, ne00] and sorted row r takes token slot[r] // top_k; without,
    src1 holds the sorted rows themselves."""
    return _ext.mul_mat_id_mxfp4(src0, ne00, ne01, src1, first, slot, top_k, acts, dst, dst_dtype, workspace, stream, flags)
