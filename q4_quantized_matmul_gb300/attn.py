"""Attention next to the projections: norms and rotation of queries and keys, the paged 4-bit cache, attention over it.

Bindings of the same names in include/q4q.h, which states the formats and formulas.  Queries, keys and
values are torch CUDA tensors [tokens, heads, head_dim] (float32, float16 or bfloat16) whose heads lie one
after another, so views of a fused projection's rows serve; caches are uint8 tensors of whole pages.
Outputs, workspaces and the stream default to new tensors and the current stream of the tensors' device.
Autograd does not see these calls; the gradients of q4q_qk_norm_rope are a call of their own, the
others have none (a cache in 4 bits is for serving).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _lib
from .mxfp4 import _check, _ext

Q4Q_ROPE_PAIRS = 0
Q4Q_ROPE_HALVES = 1


def q4q_rope_table(n_pos: int, rot: int, base: float = 10000.0, device="cuda", dst: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Cosines and sines of the positions 0 .. n_pos - 1 for rot rotated values: fp32 [n_pos, rot], rot / 2 of each."""
    if dst is None:
        dst = torch.empty((n_pos, rot), dtype=torch.float32, device=device)
    return _ext.rope_table(n_pos, rot, base, dst, stream)


def q4q_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, table: Optional[torch.Tensor] = None,
                     pos: Optional[torch.Tensor] = None, mode: int = Q4Q_ROPE_HALVES, q_dst: Optional[torch.Tensor] = None,
                     k_dst: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(q, k) with each head's row normed where it has a weight (fp32 [head_dim]) and turned by its position in the table."""
    return _ext.qk_norm_rope(q, k, q_weight, k_weight, eps, table, pos, mode, q_dst, k_dst, stream)


def q4q_qk_norm_rope_back(d_q_dst: torch.Tensor, d_k_dst: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor] = None,
                          q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          table: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None, mode: int = Q4Q_ROPE_HALVES,
                          d_q: Optional[torch.Tensor] = None, d_k: Optional[torch.Tensor] = None,
                          d_q_weight: Optional[torch.Tensor] = None, d_k_weight: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradients of q4q_qk_norm_rope: (d_q, d_k, d_q_weight, d_k_weight), None where there is no k or no weight."""
    return _ext.qk_norm_rope_back(d_q_dst, d_k_dst, q, k, q_weight, k_weight, eps, table, pos, mode, d_q, d_k, d_q_weight, d_k_weight,
                                  workspace, stream)


def q4q_qk_norm_rope_back_workspace_size(head_dim: int) -> int:
    """Bytes of workspace of q4q_qk_norm_rope_back on the current device."""
    n = ctypes.c_size_t(0)
    _check("q4q_qk_norm_rope_back_workspace_size", _lib.load().q4q_qk_norm_rope_back_workspace_size(head_dim, ctypes.byref(n)))
    return int(n.value)


@functools.lru_cache(maxsize=4096)
def q4q_kv_page_size(n_kv_heads: int, head_dim: int, page_tokens: int) -> int:
    """Bytes of a page of the cache."""
    n = ctypes.c_size_t(0)
    _check("q4q_kv_page_size", _lib.load().q4q_kv_page_size(n_kv_heads, head_dim, page_tokens, ctypes.byref(n)))
    return int(n.value)


def q4q_kv_append(cache: torch.Tensor, page_tokens: int, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                  k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, table: Optional[torch.Tensor] = None,
                  pos: Optional[torch.Tensor] = None, mode: int = Q4Q_ROPE_HALVES, stream=None) -> torch.Tensor:
    """Encode keys (normed and turned as q4q_qk_norm_rope does) and values [tokens, kv heads, head_dim] into the cache's
    slots int32 [tokens] (page * page_tokens + place); a negative slot skips its token.  Returns the cache."""
    return _ext.kv_append(cache, page_tokens, k, v, slots, k_weight, eps, table, pos, mode, stream)


def q4q_kv_get_rows(cache: torch.Tensor, page_tokens: int, n_kv_heads: int, head_dim: int, slots: torch.Tensor,
                    dst_dtype: torch.dtype = torch.float32, k_dst: Optional[torch.Tensor] = None,
                    v_dst: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cached keys and values of slots int32: two tensors [slots, kv heads, head_dim]; zeros for a negative slot."""
    return _ext.kv_get_rows(cache, page_tokens, n_kv_heads, head_dim, slots, dst_dtype, k_dst, v_dst, stream)


def q4q_kv_attn_workspace_size(n_q: int, n_q_heads: int, n_kv_heads: int, head_dim: int, n_seqs: int,
                               dtype: torch.dtype = torch.float32) -> int:
    """Bytes of workspace that serve every q4q_kv_attn on the current device with up to n_q rows of queries of dtype in up to n_seqs sequences."""
    n = ctypes.c_size_t(0)
    kind = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[dtype]
    _check("q4q_kv_attn_workspace_size", _lib.load().q4q_kv_attn_workspace_size(n_q, n_q_heads, n_kv_heads, head_dim, n_seqs, kind,
                                                                                ctypes.byref(n)))
    return int(n.value)


def q4q_kv_attn(q: torch.Tensor, cache: torch.Tensor, page_tokens: int, n_kv_heads: int, pages: torch.Tensor, kv_len: torch.Tensor,
                first: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = True, window: int = 0,
                dst: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Attention of q [rows, query heads, head_dim] over the cache, like q.

    pages int32 [sequences, pages of one]: the pages of each sequence's tokens; kv_len int32 [sequences]: its cached
    tokens, those of the rows among them; first int32 [sequences + 1]: its rows of q (None: one row each).  scale:
    1 / sqrt(head_dim) by default.  lse: fp32 [rows, query heads], filled where given.  Rows of no sequence are left as
    they are, in a new dst undefined; dst must not overlap q."""
    return _ext.kv_attn(q, cache, page_tokens, n_kv_heads, pages, kv_len, first, scale, causal, window, dst, lse, workspace, stream, None, None)


def q4q_debug_kv_attn_timeout(q: torch.Tensor, cache: torch.Tensor, page_tokens: int, n_kv_heads: int, pages: torch.Tensor,
                              kv_len: torch.Tensor, limit_ns: int, first: Optional[torch.Tensor] = None, path: int = 0) -> torch.Tensor:
    """q4q_kv_attn on one kernel (path 0: warp-level MMAs, 1: tcgen05, 16-bit types), its first CTA's first hand-off left out
    and every wait bounded by limit_ns: q4q_device_status() then reports Q4Q_ERR_TIMEOUT (6) and the result is incomplete."""
    return _ext.kv_attn(q, cache, page_tokens, n_kv_heads, pages, kv_len, first, None, True, 0, None, None, None, None, path, limit_ns)
