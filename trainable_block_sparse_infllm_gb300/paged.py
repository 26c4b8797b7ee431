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
_append = _lib.lib.infllmv2_paged_append_kv
_attn = _lib.lib.infllmv2_paged_attn_decode
_evict = _lib.lib.infllmv2_paged_evict


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
        self.scale = self.head_dim ** -0.5
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
        self._new_strides = (None, None)


# Each call's arguments are looked at in one expression; only where it fails do
# the functions named _refuse_* find out what is wrong.  get_device() is a
# tensor's device index without a device object around it, -1 on the CPU.

def _stream(cache: PagedCache, stream) -> int:
    """The stream's handle; the launch goes to the current device, which must hold the pages."""
    if torch._C._cuda_getDevice() != cache.index:
        raise _bad(f"the cache lives on {cache.device}, which is not the current CUDA device")
    if stream is None:
        # The current stream's handle without the Stream object around it (0.1 us instead of 3).
        return torch._C._cuda_getCurrentRawStream(cache.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _refuse_table(cache: PagedCache, page_table: torch.Tensor, **ints: torch.Tensor | None) -> None:
    t = page_table
    if t.dim() != 2 or t.dtype is not torch.int32 or not t.is_contiguous() or t.get_device() != cache.index:
        raise _bad(f"page_table must be contiguous int32 [batch, max_pages] on {cache.device}")
    for name, t in ints.items():
        if t is None and name in ("n_new", "seq_lens"):
            continue
        if t is None or t.dtype is not torch.int32 or t.shape != page_table.shape[:1] or not t.is_contiguous() or \
                t.get_device() != cache.index:
            raise _bad(f"{name} must be contiguous int32 [{page_table.shape[0]}] on {cache.device}")


def _optional_ints(cache: PagedCache, t: torch.Tensor | None, batch: int) -> bool:
    return t is None or (t.dtype is torch.int32 and t.dim() == 1 and t.numel() == batch and t.is_contiguous() and
                         t.get_device() == cache.index)


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
    index, dtype, shape = cache.index, cache.dtype, k_new.shape
    if page_table.dim() != 2 or page_table.dtype is not torch.int32 or not page_table.is_contiguous() or \
            page_table.get_device() != index:
        _refuse_table(cache, page_table)
    batch, max_pages = page_table.shape
    if not (kv_lens.dtype is torch.int32 and kv_lens.dim() == 1 and kv_lens.numel() == batch and
            kv_lens.is_contiguous() and kv_lens.get_device() == index and _optional_ints(cache, n_new, batch) and
            _optional_ints(cache, seq_lens, batch)):
        _refuse_table(cache, page_table, kv_lens=kv_lens, n_new=n_new, seq_lens=seq_lens)
    if len(shape) != 4 or shape != v_new.shape or shape[0] != batch or shape[1] != cache.n_kv_heads or \
            shape[3] != cache.head_dim:
        raise _bad("k_new and v_new must be [batch, n_kv_heads, n_q, head_dim]")
    strides = (k_new.stride(), v_new.stride())
    if k_new.dtype is not dtype or v_new.dtype is not dtype or strides[0][3] != 1 or strides[1][3] != 1:
        raise _bad("k_new and v_new must have the cache's type and rows of consecutive values")
    if k_new.get_device() != index or v_new.get_device() != index:
        for t in (k_new, v_new):
            if t.get_device() != index and (t.is_cuda or not t.is_pinned()):
                raise _bad(f"k_new and v_new must live on {cache.device} or in pinned host memory")
    # A loop's appends have the same strides: no new array each time.  The pair is read once and never
    # changed, so that calls from several threads each pass their own.
    kept = cache._new_strides
    if kept[0] != strides:
        cache._new_strides = kept = (strides, _Strides(*strides[0][:3], *strides[1][:3]))
    rc = _append(cache._ref, batch, max_pages, shape[2], k_new.data_ptr(), v_new.data_ptr(),
                 kept[1], page_table.data_ptr(), kv_lens.data_ptr(),
                 None if n_new is None else n_new.data_ptr(), None if seq_lens is None else seq_lens.data_ptr(),
                 _stream(cache, stream))
    if rc:
        _lib.check(rc)
    return cache


def paged_attn_decode(cache: PagedCache, q: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                      out: torch.Tensor, lse: torch.Tensor | None = None, scale: float | None = None,
                      accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """Attention of one new token per sequence, q [batch, 1, n_kv_heads * group, head_dim], over its slots.

    ``out`` like q, ``lse`` fp32 [batch, 1, heads]; ``scale`` defaults to
    1 / sqrt(head_dim).  ``accumulate``: add each slot's attention weight,
    summed over the group's heads, to the cache's weights.
    """
    index, dtype, shape = cache.index, cache.dtype, q.shape
    if page_table.dim() != 2 or page_table.dtype is not torch.int32 or not page_table.is_contiguous() or \
            page_table.get_device() != index:
        _refuse_table(cache, page_table)
    batch, max_pages = page_table.shape
    if not (kv_lens.dtype is torch.int32 and kv_lens.dim() == 1 and kv_lens.numel() == batch and
            kv_lens.is_contiguous() and kv_lens.get_device() == index):
        _refuse_table(cache, page_table, kv_lens=kv_lens)
    heads = shape[2] if len(shape) == 4 else 0
    if heads == 0 or shape[0] != batch or shape[1] != 1 or shape[3] != cache.head_dim or heads % cache.n_kv_heads != 0:
        raise _bad("q must be [batch, 1, n_kv_heads * group, head_dim]")
    if out.shape != shape or q.dtype is not dtype or out.dtype is not dtype or q.get_device() != index or \
            out.get_device() != index or not q.is_contiguous() or not out.is_contiguous():
        raise _bad("q and out must have one shape, be contiguous, of the cache's type and on its device")
    if lse is not None and (lse.dtype is not torch.float32 or lse.dim() != 3 or lse.numel() != batch * heads or
                            lse.shape[0] != batch or lse.shape[2] != heads or lse.get_device() != index or
                            not lse.is_contiguous()):
        raise _bad("lse must be contiguous fp32 [batch, 1, heads] on the cache's device")
    ws, ws_bytes = _workspace(cache, workspace)
    rc = _attn(cache._ref, batch, max_pages, heads // cache.n_kv_heads, q.data_ptr(), page_table.data_ptr(),
               kv_lens.data_ptr(), cache.scale if scale is None else scale, 1 if accumulate else 0, out.data_ptr(),
               None if lse is None else lse.data_ptr(), ws, ws_bytes, _stream(cache, stream))
    if rc:
        _lib.check(rc)
    return out, lse


def paged_evict(cache: PagedCache, page_table: torch.Tensor, kv_lens: torch.Tensor, new_lens: torch.Tensor,
                budget: int, n_init: int = 0, n_local: int = 0, seq_lens: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Keep ``budget`` slots of every (sequence, KV head) that holds more, by accumulated weight.

    The first ``n_init`` and newest ``n_local`` positions always stay.
    ``new_lens`` (int32 [batch], may be kv_lens) receives the lengths after it.
    """
    index = cache.index
    if page_table.dim() != 2 or page_table.dtype is not torch.int32 or not page_table.is_contiguous() or \
            page_table.get_device() != index:
        _refuse_table(cache, page_table)
    batch, max_pages = page_table.shape
    if kv_lens is None or new_lens is None or not (
            _optional_ints(cache, kv_lens, batch) and _optional_ints(cache, new_lens, batch) and
            _optional_ints(cache, seq_lens, batch)):
        _refuse_table(cache, page_table, kv_lens=kv_lens, new_lens=new_lens, seq_lens=seq_lens)
    ws, ws_bytes = _workspace(cache, workspace)
    rc = _evict(cache._ref, batch, max_pages, page_table.data_ptr(), kv_lens.data_ptr(), budget, n_init, n_local,
                None if seq_lens is None else seq_lens.data_ptr(), new_lens.data_ptr(), ws, ws_bytes,
                _stream(cache, stream))
    if rc:
        _lib.check(rc)
    return new_lens
