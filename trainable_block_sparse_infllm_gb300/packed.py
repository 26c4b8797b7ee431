"""Packed steps: the new tokens of several sequences one after the other.

The binding of the page tables and slot maps (``infllmv2_paged_reserve``), the
packed append, rotary positions and packed causal attention with its gradient
(include/infllmv2.h says what each computes).  A serving step in order:

    tables = alloc_page_tables(cache, batch, max_pages)                     # once
    plan = alloc_rotary_plan(rotary_dim, base=10000.0, device="cuda")       # once
    paged_reserve(tables, kv_lens, n_new, new_lens, starts, slots, positions)
    rotary(q, k, positions, plan)                                           # in place
    packed_attn(q, k, v, starts, out)                                       # prompts
    paged_append_packed(cache, k, v, slots, positions)

and ``paged_attn_decode(cache, q, tables.page_table, new_lens, out)`` where each
sequence has one new token.  Like the rest of the binding nothing here computes,
allocates (but for the ``alloc_`` functions) or synchronises.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from ._lib import InfLLMv2Error
from .paged import PagedCache, _bad, _stream as _cache_stream

_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16, torch.float32: _lib.FP32}
_reserve = _lib.lib.infllmv2_paged_reserve
_append = _lib.lib.infllmv2_paged_append_packed
_rotary = _lib.lib.infllmv2_rotary
_attn = _lib.lib.infllmv2_packed_attn
_backward = _lib.lib.infllmv2_packed_attn_backward
_byref = ctypes.byref
_int32 = torch.int32
_MAX = torch.finfo(torch.float32).max
# The C argument structures (_lib.py names their fields).
_reserve_args = struct.Struct("=6i12Q").pack
_rotary_args = struct.Struct("=8ifi6Q8q").pack
_attn_args = struct.Struct("=7if3Q6q2Q").pack
_strides2, _strides4, _strides10 = (struct.Struct("=%dq" % n).pack for n in (2, 4, 10))

# As in paged.py each call's arguments are looked at in one expression, and only
# where it fails do the functions named _refuse_* find out what is wrong.


def _on(index: int, stream) -> int:
    """The stream's handle; the launch goes to the current device, which must be `index`."""
    if torch._C._cuda_getDevice() != index:
        raise _bad(f"the tensors live on cuda:{index}, which is not the current CUDA device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _is_ints(t, index: int, n: int) -> bool:
    return t.dtype is _int32 and t.dim() == 1 and t.numel() == n and t.is_contiguous() and t.get_device() == index


def _refuse_ints(index: int, **ints) -> None:
    for name, (t, n) in ints.items():
        if t is not None and not _is_ints(t, index, n):
            raise _bad(f"{name} must be contiguous int32 [{n}] on cuda:{index}")


# ------------------------------------------------------------ pages and slots

class PageTables:
    """Which pages of a pool belong to whom: the page tables of a batch and the free pages.

    ``page_table`` int32 [batch, max_pages] and ``held`` int32 [batch]: row b
    owns its first ``held[b]`` entries; ``free_pages`` int32 [num_pages] and
    ``n_free`` int32 [1]: a stack of the free pages; ``missing`` int32 [1]: what
    the last ``paged_reserve`` lacked.  All contiguous on one CUDA device; the
    object holds them.
    """

    def __init__(self, page_table: torch.Tensor, held: torch.Tensor, free_pages: torch.Tensor, n_free: torch.Tensor,
                 missing: torch.Tensor, page_size: int):
        if not page_table.is_cuda or page_table.dtype is not torch.int32 or page_table.dim() != 2 or \
                not page_table.is_contiguous():
            raise _bad("page_table must be contiguous int32 [batch, max_pages] on a CUDA device")
        self.index = page_table.get_device()
        self.batch, self.max_pages = page_table.shape
        self.num_pages, self.page_size = free_pages.numel(), int(page_size)
        for t, n, name in ((held, self.batch, "held"), (free_pages, self.num_pages, "free_pages"),
                           (n_free, 1, "n_free"), (missing, 1, "missing")):
            if not _is_ints(t, self.index, n):
                raise _bad(f"{name} must be contiguous int32 [{n}] on cuda:{self.index}")
        self.page_table, self.held, self.free_pages = page_table, held, free_pages
        self.n_free, self.missing = n_free, missing
        self._sizes = (self.page_size, self.num_pages, self.batch, self.max_pages)
        self._arrays = (page_table.data_ptr(), held.data_ptr(), free_pages.data_ptr(), n_free.data_ptr(),
                        missing.data_ptr())
        self._lens_shape, self._starts_shape = held.shape, torch.Size([self.batch + 1])


def alloc_page_tables(cache: PagedCache, batch: int, max_pages: int) -> PageTables:
    """Empty page tables over the cache's pool: every page is free, page 0 on top."""
    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=cache.device)
    free = torch.arange(cache.num_pages - 1, -1, -1, dtype=torch.int32, device=cache.device)
    return PageTables(ints(batch, max_pages), ints(batch), free, ints(1).fill_(cache.num_pages), ints(1),
                      cache.page_size)


def paged_reserve(tables: PageTables, kv_lens: torch.Tensor, n_new: torch.Tensor, new_lens: torch.Tensor,
                  starts: torch.Tensor, slots: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                  seq_lens: torch.Tensor | None = None, stream=None) -> PageTables:
    """Take and give back pages for a step of ``n_new[b]`` tokens after ``kv_lens[b]``, and map its tokens.

    Writes ``new_lens`` (int32 [batch], may be kv_lens) and ``starts`` (int32
    [batch + 1]) and, for a step of up to their common length of tokens,
    ``slots`` and ``positions`` (int32 [tokens]).  ``seq_lens``: the tokens each
    sequence has seen before (default kv_lens).  Where pages lack,
    ``tables.missing`` says how many and the step is empty.
    """
    index, shape = tables.index, tables._lens_shape
    if not (kv_lens.dtype is _int32 and n_new.dtype is _int32 and new_lens.dtype is _int32 and
            starts.dtype is _int32 and kv_lens.shape == shape and n_new.shape == shape and new_lens.shape == shape and
            starts.shape == tables._starts_shape and kv_lens.is_contiguous() and n_new.is_contiguous() and
            new_lens.is_contiguous() and starts.is_contiguous() and kv_lens.get_device() == index and
            n_new.get_device() == index and new_lens.get_device() == index and starts.get_device() == index):
        _refuse_ints(index, kv_lens=(kv_lens, tables.batch), n_new=(n_new, tables.batch),
                     new_lens=(new_lens, tables.batch), starts=(starts, tables.batch + 1))
    seen = map_slots = map_positions = tokens = 0
    if seq_lens is not None:
        if not (seq_lens.dtype is _int32 and seq_lens.shape == shape and seq_lens.is_contiguous() and
                seq_lens.get_device() == index):
            _refuse_ints(index, seq_lens=(seq_lens, tables.batch))
        seen = seq_lens.data_ptr()
    if slots is not None:
        tokens = slots.numel()
        if not (slots.dtype is _int32 and slots.dim() == 1 and slots.is_contiguous() and slots.get_device() == index):
            _refuse_ints(index, slots=(slots, tokens))
        map_slots = slots.data_ptr() or starts.data_ptr()   # (one of no tokens has no memory, but is there)
    if positions is not None:
        tokens = tokens if slots is not None else positions.numel()
        if not (positions.dtype is _int32 and positions.dim() == 1 and positions.numel() == tokens and
                positions.is_contiguous() and positions.get_device() == index):
            _refuse_ints(index, positions=(positions, tokens))
        map_positions = positions.data_ptr() or starts.data_ptr()
    rc = _reserve(_reserve_args(*tables._sizes, tokens, 0, *tables._arrays, kv_lens.data_ptr(), n_new.data_ptr(), seen,
                                new_lens.data_ptr(), starts.data_ptr(), map_slots, map_positions), _on(index, stream))
    if rc:
        _lib.check(rc)
    return tables


def paged_append_packed(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor,
                        positions: torch.Tensor | None = None, stream=None) -> PagedCache:
    """Write a packed step's k_new / v_new [tokens, n_kv_heads, head_dim] to the pages' ``slots`` (int32 [tokens]).

    A slot below 0 is not written.  ``positions`` (int32 [tokens]) is needed
    where the cache has positions.  Any strides with consecutive values;
    pinned host tensors are accepted.
    """
    index, dtype, shape = cache.index, cache.dtype, k_new.shape
    if len(shape) != 3 or shape != v_new.shape or shape[1] != cache.n_kv_heads or shape[2] != cache.head_dim:
        raise _bad("k_new and v_new must be [tokens, n_kv_heads, head_dim]")
    tokens, k_st, v_st = shape[0], k_new.stride(), v_new.stride()
    if k_new.dtype is not dtype or v_new.dtype is not dtype or k_st[2] != 1 or v_st[2] != 1:
        raise _bad("k_new and v_new must have the cache's type and rows of consecutive values")
    if k_new.get_device() != index or v_new.get_device() != index:
        for t in (k_new, v_new):
            if t.get_device() != index and (t.is_cuda or not t.is_pinned()):
                raise _bad(f"k_new and v_new must live on {cache.device} or in pinned host memory")
    if not (slots.dtype is _int32 and slots.dim() == 1 and slots.numel() == tokens and slots.is_contiguous() and
            slots.get_device() == index):
        _refuse_ints(index, slots=(slots, tokens))
    where = None
    if positions is not None:
        if not (positions.dtype is _int32 and positions.dim() == 1 and positions.numel() == tokens and
                positions.is_contiguous() and positions.get_device() == index):
            _refuse_ints(index, positions=(positions, tokens))
        where = positions.data_ptr()
    rc = _append(cache._ref, tokens, k_new.data_ptr(), v_new.data_ptr(),
                 _strides4(k_st[0], k_st[1], v_st[0], v_st[1]), slots.data_ptr(), where, _cache_stream(cache, stream))
    if rc:
        _lib.check(rc)
    return cache


# --------------------------------------------------------------------- rotary

class RotaryPlan:
    """The frequencies of rotary positions: ``turns`` int64 [rotary_dim / 2] on a CUDA device and ``scale``."""

    def __init__(self, turns: torch.Tensor, scale: float):
        if not turns.is_cuda or turns.dtype is not torch.int64 or turns.dim() != 1 or not turns.is_contiguous():
            raise _bad("turns must be contiguous int64 [rotary_dim / 2] on a CUDA device")
        if not abs(scale) < _MAX:
            raise _bad("scale must be finite in fp32")
        self.turns, self.scale, self.rotary_dim, self.index = turns, scale, 2 * turns.numel(), turns.get_device()
        self._ptr = turns.data_ptr()


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: int = _lib.ROTARY_PLAIN, factor: float = 1.0,
                       original_len: int = 0, fast_turns: float = 32.0, slow_turns: float = 1.0,
                       factors=None) -> tuple[list[int], float]:
    """2^64 times the turns per position of each pair, and the factor of the turned values (host code).

    ``scaling``: ROTARY_PLAIN, _LINEAR, _BASE, _PARTS or _FACTORS; ``factors``
    are rotary_dim / 2 divisors for the last.
    """
    if factors is not None and len(factors) != rotary_dim // 2:
        raise _bad(f"factors must have rotary_dim / 2 = {rotary_dim // 2} entries (got {len(factors)})")
    divisors = None if factors is None else (ctypes.c_double * len(factors))(*factors)
    config = _lib.RotaryConfig(rotary_dim=rotary_dim, scaling=scaling, base=base, factor=factor,
                               original_len=original_len, fast_turns=fast_turns, slow_turns=slow_turns,
                               factors=divisors)
    turns, scale = (ctypes.c_uint64 * max(rotary_dim // 2, 1))(), ctypes.c_float()
    _lib.check(_lib.lib.infllmv2_rotary_frequencies(_byref(config), turns, _byref(scale)))
    return list(turns), float(scale.value)


def alloc_rotary_plan(rotary_dim: int, base: float = 10000.0, scaling: int = _lib.ROTARY_PLAIN, factor: float = 1.0,
                      original_len: int = 0, fast_turns: float = 32.0, slow_turns: float = 1.0, factors=None,
                      device=None) -> RotaryPlan:
    """``rotary_frequencies`` as a plan on a CUDA device."""
    turns, scale = rotary_frequencies(rotary_dim, base, scaling, factor, original_len, fast_turns, slow_turns, factors)
    signed = [t - (1 << 64) if t >> 63 else t for t in turns]
    return RotaryPlan(torch.tensor(signed, dtype=torch.int64, device=device or "cuda"), scale)


def _refuse_rotary(x: torch.Tensor, out: torch.Tensor, name: str, q: torch.Tensor) -> None:
    if x.dim() != 3 or out.shape != x.shape or x.shape[0] != q.shape[0] or x.shape[2] != q.shape[2]:
        raise _bad(f"{name} and its output must be [tokens, heads, head_dim], of one head_dim and count of tokens")
    if x.dtype is not q.dtype or out.dtype is not q.dtype or x.get_device() != q.get_device() or \
            out.get_device() != q.get_device():
        raise _bad(f"{name} and its output must have q's type and live on its device")
    if x.stride(2) != 1 or out.stride(2) != 1:
        raise _bad(f"{name}: the values of a head must be consecutive")


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, plan: RotaryPlan,
           q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, interleaved: bool = False,
           transpose: bool = False, stream=None):
    """Turn the first plan.rotary_dim values of every head of q and k [tokens, heads, head_dim] by their positions.

    bf16, fp16 or fp32, any strides with consecutive values; ``q_out`` and
    ``k_out`` default to q and k (in place).  ``positions`` int32 [tokens].
    ``interleaved``: pairs are neighbours instead of half the dimension apart.
    ``transpose``: the gradient of the inputs from that of the outputs.
    """
    index, dtype, shape = q.get_device(), q.dtype, q.shape
    kind = _DTYPES.get(dtype)
    if kind is None or index < 0 or len(shape) != 3:
        raise _bad("q must be bf16, fp16 or fp32 [tokens, heads, head_dim] on a CUDA device")
    tokens, heads, dim = shape
    if plan.index != index or not (positions.dtype is _int32 and positions.dim() == 1 and
                                   positions.numel() == tokens and positions.is_contiguous() and
                                   positions.get_device() == index):
        raise _bad(f"positions must be contiguous int32 [{tokens}], and the plan's frequencies, on cuda:{index}")
    q_out = q if q_out is None else q_out
    st, so = q.stride(), q_out.stride()
    if q_out.shape != shape or q_out.dtype is not dtype or q_out.get_device() != index or st[2] != 1 or so[2] != 1:
        _refuse_rotary(q, q_out, "q", q)
    k_in = k_to = k_heads = 0
    kt = ko = (0, 0)
    if k is not None:
        k_out = k if k_out is None else k_out
        k_shape, kt, ko = k.shape, k.stride(), k_out.stride()
        if len(k_shape) != 3 or k_out.shape != k_shape or k_shape[0] != tokens or k_shape[2] != dim or \
                k.dtype is not dtype or k_out.dtype is not dtype or k.get_device() != index or \
                k_out.get_device() != index or kt[2] != 1 or ko[2] != 1:
            _refuse_rotary(k, k_out, "k", q)
        k_in, k_to, k_heads = k.data_ptr(), k_out.data_ptr(), k_shape[1]
        if k_heads == 0:
            raise _bad("k has no heads")
    rc = _rotary(_rotary_args(kind, tokens, dim, plan.rotary_dim, heads, k_heads, 1 if interleaved else 0,
                              1 if transpose else 0, plan.scale, 0, positions.data_ptr(), plan._ptr, q.data_ptr(),
                              q_out.data_ptr(), k_in, k_to, st[0], st[1], so[0], so[1], kt[0], kt[1], ko[0], ko[1]),
                 _on(index, stream))
    if rc:
        _lib.check(rc)
    return q_out, k_out


# ------------------------------------------------------------------ attention

def _inputs(q, k, v, q_starts, k_starts, scale):
    """The argument structure of an attention call."""
    q_shape, k_shape, dtype, index = q.shape, k.shape, q.dtype, q.get_device()
    if len(q_shape) != 3 or len(k_shape) != 3 or v.shape != k_shape or q_shape[2] != k_shape[2] or \
            k_shape[1] == 0 or q_shape[1] == 0 or q_shape[1] % k_shape[1] != 0:
        raise _bad("q must be [tokens, n_kv_heads * group, head_dim], k and v [tokens, n_kv_heads, head_dim]")
    if (dtype is not torch.bfloat16 and dtype is not torch.float16) or k.dtype is not dtype or v.dtype is not dtype:
        raise _bad("q, k and v must all be bf16 or all fp16")
    if index < 0 or k.get_device() != index or v.get_device() != index:
        raise _bad("q, k and v must live on one CUDA device")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if qs[2] != 1 or ks[2] != 1 or vs[2] != 1:
        raise _bad("the values of a head must be consecutive")
    if scale is not None and not abs(scale) < _MAX:
        raise _bad("scale must be finite in fp32")
    batch = q_starts.numel() - 1
    if batch < 1 or not _is_ints(q_starts, index, batch + 1) or \
            not (k_starts is None or _is_ints(k_starts, index, batch + 1)):
        raise _bad(f"q_starts and k_starts must be contiguous int32 [batch + 1] on cuda:{index}")
    return _attn_args(_DTYPES[dtype], batch, k_shape[1], q_shape[1] // k_shape[1], q_shape[2], q_shape[0], k_shape[0],
                      q_shape[2] ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                      qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], q_starts.data_ptr(),
                      0 if k_starts is None else k_starts.data_ptr())


def _like(x: torch.Tensor, y: torch.Tensor, name: str):
    """The strides of `x`, which must be of y's shape, type and device."""
    if x.shape != y.shape or x.dtype is not y.dtype or x.get_device() != y.get_device():
        raise _bad(f"{name} must have the shape, type and device of the tensor it belongs to")
    st = x.stride()
    if st[2] != 1:
        raise _bad(f"{name}: the values of a head must be consecutive")
    return st


def _sums(lse: torch.Tensor, q: torch.Tensor) -> int:
    if lse.dtype is not torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous() or \
            lse.get_device() != q.get_device():
        raise _bad("lse must be contiguous fp32 [tokens, heads] on q's device")
    return lse.data_ptr()


def packed_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor, out: torch.Tensor,
                lse: torch.Tensor | None = None, k_starts: torch.Tensor | None = None, scale: float | None = None,
                stream=None):
    """Causal attention of packed sequences: q, out [tokens, n_kv_heads * group, head_dim], k and v their keys' rows.

    ``q_starts`` int32 [batch + 1]; ``k_starts`` where the sequences have more
    (earlier) keys than queries; ``lse`` fp32 [tokens, heads], which the
    gradient needs.  ``scale`` defaults to 1 / sqrt(head_dim).  Rows of no
    sequence are left as they were.
    """
    args = _inputs(q, k, v, q_starts, k_starts, scale)
    st = _like(out, q, "out")
    rc = _attn(args, out.data_ptr(), _strides2(st[0], st[1]),
               None if lse is None else _sums(lse, q), _on(q.get_device(), stream))
    if rc:
        _lib.check(rc)
    return out, lse


def packed_workspace_size(q: torch.Tensor) -> int:
    """Bytes of workspace of ``packed_attn_backward`` for queries like q."""
    return 8 * q.shape[0] * q.shape[1]


def alloc_packed_workspace(q: torch.Tensor) -> torch.Tensor:
    """A workspace for ``packed_attn_backward`` with queries of q's shape."""
    return torch.empty(max(packed_workspace_size(q), 16), dtype=torch.uint8, device=q.device)


def packed_attn_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor,
                         out: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor, dq: torch.Tensor,
                         dk: torch.Tensor, dv: torch.Tensor, workspace: torch.Tensor,
                         k_starts: torch.Tensor | None = None, scale: float | None = None, stream=None):
    """dq, dk, dv (of q's type) of ``packed_attn`` for the upstream gradient ``dout`` of ``out``.

    ``out`` and ``lse`` are the forward call's on the same arguments.
    """
    args = _inputs(q, k, v, q_starts, k_starts, scale)
    strides = _strides10(*_like(out, q, "out")[:2], *_like(dout, q, "dout")[:2], *_like(dq, q, "dq")[:2],
                         *_like(dk, k, "dk")[:2], *_like(dv, v, "dv")[:2])
    index = q.get_device()
    if not workspace.is_contiguous() or workspace.get_device() != index:
        raise _bad(f"workspace must be contiguous on cuda:{index}")
    rc = _backward(args, out.data_ptr(), _sums(lse, q), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                   dv.data_ptr(), strides, workspace.data_ptr(), workspace.nbytes, _on(index, stream))
    if rc:
        _lib.check(rc)
    return dq, dk, dv


__all__ = ["PageTables", "alloc_page_tables", "paged_reserve", "paged_append_packed", "RotaryPlan",
           "rotary_frequencies", "alloc_rotary_plan", "rotary", "packed_attn", "packed_workspace_size",
           "alloc_packed_workspace", "packed_attn_backward", "InfLLMv2Error"]
