"""A paged key-value cache: append, single-token attention, eviction.

The binding of the ``infllmv2_paged_*`` functions (include/infllmv2.h says
what each computes).  ``PagedCache`` describes a pool of pages once; the calls
take it with the page table and the lengths of the sequences at hand:

    cache = PagedCache(k_pages, v_pages, weights, positions)
    ws = alloc_paged_workspace(cache, page_table, OP_PAGED_DECODE, group_size)
    paged_append_kv(cache, k_new, v_new, page_table, kv_lens)
    paged_attn_decode(cache, q, page_table, kv_lens, out, accumulate=True, workspace=ws)
    paged_evict(cache, page_table, kv_lens, new_lens, budget, workspace=ws_evict)

Like the rest of the binding nothing here computes, allocates (but for the
``alloc_`` function) or synchronises: the calls check their arguments and
enqueue on the current stream.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import InfLLMv2Error

_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16}
_Strides = ctypes.c_int64 * 6


def _bad(message: str):
    return InfLLMv2Error(_lib.INVALID_ARGUMENT, message)


class PagedCache:
    """A pool of pages.

    ``k_pages`` and ``v_pages``: bf16 or fp16 [num_pages, n_kv_heads,
    page_size, head_dim] on one CUDA device, any strides as long as a row's
    values are consecutive (a transposed view of token-major storage, or
    ``buffer[:, 0]`` and ``buffer[:, 1]`` of one buffer for both).
    ``weights`` (fp32) and ``positions`` (int32): contiguous [num_pages,
    n_kv_heads, page_size], or None; ``paged_attn_decode(accumulate=True)``
    needs the first and ``paged_evict`` both.  The object holds the tensors.
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, weights: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
            raise _bad("k_pages and v_pages must have one shape [num_pages, n_kv_heads, page_size, head_dim]")
        if k_pages.dtype not in _DTYPES or v_pages.dtype != k_pages.dtype:
            raise _bad("k_pages and v_pages must both be bf16 or both fp16")
        if not k_pages.is_cuda or v_pages.device != k_pages.device:
            raise _bad("k_pages and v_pages must live on one CUDA device")
        for t in (k_pages, v_pages):
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise _bad("the values of a row must be consecutive")
        for t, dtype, name in ((weights, torch.float32, "weights"), (positions, torch.int32, "positions")):
            if t is None:
                continue
            if t.shape != k_pages.shape[:3] or t.dtype != dtype or not t.is_contiguous() or t.device != k_pages.device:
                raise _bad(f"{name} must be contiguous {dtype} [num_pages, n_kv_heads, page_size] on the pages' device")
        self.k_pages, self.v_pages, self.weights, self.positions = k_pages, v_pages, weights, positions
        self.num_pages, self.n_kv_heads, self.page_size, self.head_dim = k_pages.shape
        self.dtype, self.device, self.index = k_pages.dtype, k_pages.device, k_pages.get_device()
        self.struct = _lib.PagedCacheStruct(
            dtype=_DTYPES[k_pages.dtype], n_kv_heads=self.n_kv_heads, head_dim=self.head_dim,
            page_size=self.page_size, num_pages=self.num_pages,
            k_strides=k_pages.stride()[:3],
            v_strides=v_pages.stride()[:3],
            k_pages=k_pages.data_ptr(), v_pages=v_pages.data_ptr(),
            weights=weights.data_ptr() if weights is not None else None,
            positions=positions.data_ptr() if positions is not None else None)
        self._ref = ctypes.byref(self.struct)


def _stream(cache: PagedCache, stream) -> int:
    """The stream's handle; the launch goes to the current device, which must hold the pages."""
    index = cache.index
    if torch.cuda.current_device() != index:
        raise _bad(f"the cache lives on {cache.device}, which is not the current CUDA device")
    if stream is None:
        # The current stream's handle without the Stream object around it (0.1 us instead of 3).
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# get_device() is the device's index without a device object around it, -1 on the CPU.

def _ints(cache: PagedCache, t: torch.Tensor | None, batch: int, name: str):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.dim() != 1 or t.numel() != batch or not t.is_contiguous() or \
            t.get_device() != cache.index:
        raise _bad(f"{name} must be contiguous int32 [{batch}] on {cache.device}")
    return t.data_ptr()


def _table(cache: PagedCache, t: torch.Tensor):
    if t.dim() != 2 or t.dtype is not torch.int32 or not t.is_contiguous() or t.get_device() != cache.index:
        raise _bad(f"page_table must be contiguous int32 [batch, max_pages] on {cache.device}")
    batch, max_pages = t.shape
    return batch, max_pages, t.data_ptr()


def _workspace(cache: PagedCache, workspace: torch.Tensor | None):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous() or workspace.get_device() != cache.index:
        raise _bad(f"workspace must be contiguous on {cache.device}")
    return workspace.data_ptr(), workspace.nbytes


def paged_workspace_size(cache: PagedCache, batch: int, max_pages: int, op: int, group_size: int = 1) -> int:
    """Bytes of workspace of OP_PAGED_DECODE (group_size query heads per KV head) or OP_PAGED_EVICT."""
    return int(_lib.lib.infllmv2_paged_workspace_size(cache._ref, batch, max_pages, group_size, op))


def alloc_paged_workspace(cache: PagedCache, page_table: torch.Tensor, op: int, group_size: int = 1) -> torch.Tensor:
    """A workspace for calls with page tables of this shape."""
    n = paged_workspace_size(cache, page_table.shape[0], page_table.shape[1], op, group_size)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def paged_append_kv(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, page_table: torch.Tensor,
                    kv_lens: torch.Tensor, n_new: torch.Tensor | None = None, seq_lens: torch.Tensor | None = None,
                    stream=None) -> PagedCache:
    """Write the newest tokens' k_new / v_new [batch, n_kv_heads, n_q, head_dim] into the pages.

    Sequence b's first ``n_new[b]`` tokens (default: all n_q) go to slots
    ``kv_lens[b] - n_new[b]`` onward; ``kv_lens`` already counts them, as does
    ``seq_lens``, the tokens each sequence has seen (default: kv_lens).  Any
    strides with consecutive values; pinned host tensors are accepted.
    """
    batch, max_pages, table = _table(cache, page_table)
    shape = k_new.shape
    if len(shape) != 4 or shape != v_new.shape or shape[0] != batch or shape[1] != cache.n_kv_heads or \
            shape[3] != cache.head_dim:
        raise _bad("k_new and v_new must be [batch, n_kv_heads, n_q, head_dim]")
    kb, kh, kt, kd = k_new.stride()
    vb, vh, vt, vd = v_new.stride()
    for t, unit in ((k_new, kd), (v_new, vd)):
        if t.dtype is not cache.dtype or unit != 1:
            raise _bad("k_new and v_new must have the cache's type and rows of consecutive values")
        if t.get_device() != cache.index and (t.is_cuda or not t.is_pinned()):
            raise _bad(f"k_new and v_new must live on {cache.device} or in pinned host memory")
    _lib.check(_lib.lib.infllmv2_paged_append_kv(
        cache._ref, batch, max_pages, shape[2], k_new.data_ptr(), v_new.data_ptr(), _Strides(kb, kh, kt, vb, vh, vt), table,
        _ints(cache, kv_lens, batch, "kv_lens"), _ints(cache, n_new, batch, "n_new"),
        _ints(cache, seq_lens, batch, "seq_lens"), _stream(cache, stream)))
    return cache


def paged_attn_decode(cache: PagedCache, q: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                      out: torch.Tensor, lse: torch.Tensor | None = None, scale: float | None = None,
                      accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """Attention of one new token per sequence, q [batch, 1, n_kv_heads * group, head_dim], over its slots.

    ``out`` like q, ``lse`` fp32 [batch, 1, heads]; ``scale`` defaults to
    1 / sqrt(head_dim).  ``accumulate``: add each slot's attention weight,
    summed over the group's heads, to the cache's weights.
    """
    batch, max_pages, table = _table(cache, page_table)
    shape = q.shape
    heads = shape[2] if len(shape) == 4 else 0
    if heads == 0 or shape[0] != batch or shape[1] != 1 or shape[3] != cache.head_dim or heads % cache.n_kv_heads != 0:
        raise _bad("q must be [batch, 1, n_kv_heads * group, head_dim]")
    if out.shape != shape:
        raise _bad("out must have q's shape")
    for t in (q, out):
        if t.dtype is not cache.dtype or t.get_device() != cache.index or not t.is_contiguous():
            raise _bad("q and out must be contiguous, of the cache's type and on its device")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (batch, 1, heads) or
                            lse.get_device() != cache.index or not lse.is_contiguous()):
        raise _bad("lse must be contiguous fp32 [batch, 1, heads] on the cache's device")
    ws, ws_bytes = _workspace(cache, workspace)
    _lib.check(_lib.lib.infllmv2_paged_attn_decode(
        cache._ref, batch, max_pages, heads // cache.n_kv_heads, q.data_ptr(), table,
        _ints(cache, kv_lens, batch, "kv_lens"), cache.head_dim ** -0.5 if scale is None else scale,
        1 if accumulate else 0, out.data_ptr(), lse.data_ptr() if lse is not None else None, ws, ws_bytes,
        _stream(cache, stream)))
    return out, lse


def paged_evict(cache: PagedCache, page_table: torch.Tensor, kv_lens: torch.Tensor, new_lens: torch.Tensor,
                budget: int, n_init: int = 0, n_local: int = 0, seq_lens: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Keep ``budget`` slots of every (sequence, KV head) that holds more, by accumulated weight.

    The first ``n_init`` and newest ``n_local`` positions always stay.
    ``new_lens`` (int32 [batch], may be kv_lens) receives the lengths after it.
    """
    batch, max_pages, table = _table(cache, page_table)
    if new_lens is None:
        raise _bad("new_lens is required")
    ws, ws_bytes = _workspace(cache, workspace)
    _lib.check(_lib.lib.infllmv2_paged_evict(
        cache._ref, batch, max_pages, table, _ints(cache, kv_lens, batch, "kv_lens"), budget, n_init, n_local,
        _ints(cache, seq_lens, batch, "seq_lens"), _ints(cache, new_lens, batch, "new_lens"), ws, ws_bytes,
        _stream(cache, stream)))
    return new_lens
