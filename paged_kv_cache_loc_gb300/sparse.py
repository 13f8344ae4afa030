"""Python binding of the sparse decode path and of the tables it reads
(include/pkv.h: pkv_build_tables, pkv_page_bounds, pkv_select_pages,
pkv_paged_decode_selected, pkv_sparse_decode_step).

Argument marshalling only, like ops.py.  These calls run once per layer and
step, so the shapes are checked with plain comparisons and the descriptors are
filled in one constructor call.  They work on the device of the cache, whatever
the current one is; outputs that are not given are allocated for the stream
that the kernels run on.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import PkvKVCache, PkvPages, PkvTables, check
from .ops import KVCache, Workspace, _DTYPES, _need


def _ptr(t: torch.Tensor, name: str, dtype, index: int) -> int:
    """The address of a contiguous tensor of `dtype` on CUDA device `index`,
    or in pinned host memory (as in ops._need)."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return _need(t, name, dtype, torch.device("cuda", index))


def _i32(t: Optional[torch.Tensor], name: str, index: int, n: int) -> Optional[int]:
    """The address of an int32 array of n elements; None stays None."""
    if t is None:
        return None
    p = _ptr(t, name, torch.int32, index)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return p


@dataclasses.dataclass
class SparsePages:
    """The page table of a cache and what its pages' keys are bounded by
    (struct pkv_pages).  req_to_page: int32 [num_reqs, max_pages] of physical
    pages (runs of page_size consecutive slots); page_bounds: [n_layers, size //
    page_size, n_kv_heads, 2, head_dim] of the cache's dtype; top_k: pages
    selected per query and kv head, the context's n_first first and n_last last
    ones among them."""
    page_bounds: Optional[torch.Tensor]
    req_to_page: torch.Tensor
    page_size: int
    top_k: int
    n_first: int = 1
    n_last: int = 1

    @classmethod
    def for_cache(cls, cache: KVCache, req_to_page: torch.Tensor, page_size: int, top_k: int,
                  n_first: int = 1, n_last: int = 1) -> "SparsePages":
        """With page_bounds allocated for the cache's pool."""
        n_layers, size, n_kv_heads, head_dim = cache.k_buffer.shape
        bounds = torch.zeros(n_layers, size // page_size, n_kv_heads, 2, head_dim,
                             dtype=cache.k_buffer.dtype, device=cache.device)
        return cls(bounds, req_to_page, page_size, top_k, n_first, n_last)

    def c_struct(self, cache: KVCache) -> PkvPages:
        kb, t, bounds, ps = cache.k_buffer, self.req_to_page, self.page_bounds, self.page_size
        index = kb.get_device()
        if t.dim() != 2:
            raise ValueError("req_to_page must be [num_reqs, max_pages]")
        if ps < 1:
            raise ValueError("page_size must be positive")
        if bounds is not None:
            n_layers, size, n_kv_heads, head_dim = kb.shape
            if bounds.shape != (n_layers, size // ps, n_kv_heads, 2, head_dim):
                raise ValueError("page_bounds must be [n_layers, size // page_size, n_kv_heads, 2, head_dim]")
            bounds = _ptr(bounds, "page_bounds", kb.dtype, index)
        return PkvPages(bounds, _ptr(t, "req_to_page", torch.int32, index), t.shape[1], ps, self.top_k, self.n_first,
                        self.n_last)


def _cache(cache: KVCache, table: torch.Tensor, table_ptr: int, max_ctx_len: int, n_new: int,
           decode: bool) -> Tuple[PkvKVCache, int]:
    """The descriptor of a cache whose request rows are those of `table`
    (already checked, at table_ptr)."""
    kb, vb, rows, lens = cache.k_buffer, cache.v_buffer, cache.req_pool_indices, cache.seq_lens
    dtype = kb.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported storage dtype {dtype}")
    shape = kb.shape
    if len(shape) != 4 or vb.shape != shape:
        raise ValueError("k_buffer/v_buffer must both be [n_layers, size, n_kv_heads, head_dim]")
    index = kb.get_device()
    if index < 0:
        raise ValueError("k_buffer must be a CUDA tensor (there is no CPU path)")
    batch = rows.numel()
    if lens is not None:
        lens = _i32(lens, "seq_lens", index, batch)
    elif decode:
        raise ValueError("seq_lens is needed")
    n_layers, size, n_kv_heads, head_dim = shape
    return PkvKVCache(
        _ptr(kb, "k_buffer", dtype, index), _ptr(vb, "v_buffer", dtype, index), code, n_layers, n_kv_heads,
        head_dim, size, table_ptr, table.shape[0], max_ctx_len,
        _ptr(rows, "req_pool_indices", torch.int32, index), lens, None, None,
        _slots(cache.out_cache_loc, index, n_new) if n_new else None, batch, int(cache.max_len)), index


def _slots(loc: Optional[torch.Tensor], index: int, n_new: int) -> int:
    """The address of out_cache_loc, which may be longer than what is written."""
    p = _ptr(loc, "out_cache_loc", torch.int32, index)
    if loc.numel() < n_new:
        raise ValueError(f"out_cache_loc must have {n_new} elements at least, got {loc.numel()}")
    return p


def _rows(t: torch.Tensor, name: str, c: PkvKVCache, dtype, index: int, n: int, heads: int) -> int:
    """The address of [n, heads, head_dim] rows of the cache's dtype."""
    if t.shape != (n, heads, c.head_dim):
        raise ValueError(f"{name} must be [{n}, {heads}, {c.head_dim}], got {list(t.shape)}")
    return _ptr(t, name, dtype, index)


def _heads(q: torch.Tensor) -> int:
    if q.dim() != 3:
        raise ValueError(f"q must be [batch, n_heads, head_dim], got {list(q.shape)}")
    return q.shape[1]


def _lists(sel: torch.Tensor, counts: torch.Tensor, c: PkvKVCache, top_k: int, index: int) -> Tuple[int, int]:
    n = c.batch * c.n_kv_heads
    return _i32(sel, "sel", index, n * top_k), _i32(counts, "sel_counts", index, n)


def _workspace(ws: Optional[Workspace], index: int):
    if ws is None:
        return None
    if ws.buffer.get_device() != index:
        raise ValueError(f"workspace is on {ws.buffer.device}, expected cuda:{index}")
    return ctypes.byref(ws.desc)


# the handle of a device's current stream, without the object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, index: int, stream, *args) -> None:
    """Calls the library's `name` on the cache's device with the stream's
    handle; None is the device's current stream."""
    fn = getattr(_lib._lib or _lib.load(), name)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status:
        check(status, name)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output, allocated for the stream that the kernels run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def build_tables(cache: KVCache, req_to_page: torch.Tensor, page_size: int, free_pages: torch.Tensor,
                 free_start: torch.Tensor, free_end: torch.Tensor,
                 positions: Optional[torch.Tensor] = None, q_lens: Optional[torch.Tensor] = None,
                 token_table: bool = True, stream=None) -> None:
    """A step's tables from the lengths cache.seq_lens (the q_lens new tokens
    included; None: one new token for each entry that is not empty).  New pages
    are taken from free_pages[free_start[0]:] into req_to_page, and free_end[0]
    becomes the next free place.  Writes cache.out_cache_loc, positions,
    cache.kv_indptr and cache.qo_indptr (each where it is given), and the new
    tokens' entries of cache.req_to_token unless token_table is False.  Tokens
    beyond out_cache_loc's length are an error on the device; entries of
    out_cache_loc behind the last new token stay as they are."""
    if req_to_page.dim() != 2 or cache.req_to_token.dim() != 2:
        raise ValueError("req_to_page must be [num_reqs, max_pages], req_to_token [num_reqs, max_ctx_len]")
    if token_table and cache.req_to_token.shape[0] != req_to_page.shape[0]:
        raise ValueError("req_to_page and req_to_token must have the same rows")
    loc = cache.out_cache_loc
    n_new = 0 if loc is None else loc.numel()
    c, index = _cache(cache, req_to_page, _ptr(req_to_page, "req_to_page", torch.int32, cache.k_buffer.get_device()), cache.req_to_token.shape[1], n_new, True)
    t = PkvTables(
        _i32(q_lens, "q_lens", index, c.batch), c.req_to_token, req_to_page.shape[1], int(page_size),
        _ptr(free_pages, "free_pages", torch.int32, index), _i32(free_start, "free_start", index, 1),
        _i32(free_end, "free_end", index, 1), free_pages.numel(), n_new,
        _i32(cache.kv_indptr, "kv_indptr", index, c.batch + 1),
        _i32(cache.qo_indptr, "qo_indptr", index, c.batch + 1),
        _i32(positions, "positions", index, n_new), c.out_cache_loc,
        _ptr(cache.req_to_token, "req_to_token", torch.int32, index) if token_table else None)
    _call("pkv_build_tables", index, stream, ctypes.byref(c), ctypes.byref(t))


def page_bounds(cache: KVCache, layer_id: int, pages: SparsePages, n_new: Optional[int] = None,
                stream=None) -> None:
    """Bring pages.page_bounds up to date with the keys written to the slots
    cache.out_cache_loc[:n_new] (None: all of them) of the layer."""
    if cache.out_cache_loc is None or pages.page_bounds is None:
        raise ValueError("out_cache_loc and page_bounds are needed")
    if n_new is None:
        n_new = cache.out_cache_loc.numel()
    pg = pages.c_struct(cache)
    c, index = _cache(cache, pages.req_to_page, pg.req_to_page, 0, n_new, False)
    _call("pkv_page_bounds", index, stream, ctypes.byref(c), layer_id, ctypes.byref(pg), n_new)


def select_workspace_bytes(batch: int, n_kv_heads: int, max_len: int, page_size: int) -> int:
    """Workspace bytes that select_pages and sparse_decode_step need."""
    return _lib.load().pkv_select_workspace_bytes(batch, n_kv_heads, max_len, page_size)


def select_pages(cache: KVCache, layer_id: int, pages: SparsePages, q: torch.Tensor,
                 sel: Optional[torch.Tensor] = None, sel_counts: Optional[torch.Tensor] = None,
                 workspace: Optional[Workspace] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The pages that each query of q [batch, n_heads, head_dim] attends to:
    sel int32 [batch, n_kv_heads, top_k] (logical pages, ascending, then -1)
    and sel_counts int32 [batch, n_kv_heads]."""
    pg = pages.c_struct(cache)
    c, index = _cache(cache, pages.req_to_page, pg.req_to_page, 0, 0, True)
    if sel is None:
        sel = _empty((c.batch, c.n_kv_heads, pages.top_k), torch.int32, cache.k_buffer.device, stream)
    if sel_counts is None:
        sel_counts = _empty((c.batch, c.n_kv_heads), torch.int32, cache.k_buffer.device, stream)
    _call("pkv_select_pages", index, stream, ctypes.byref(c), layer_id, ctypes.byref(pg),
            _rows(q, "q", c, cache.k_buffer.dtype, index, c.batch, _heads(q)), q.shape[1],
            *_lists(sel, sel_counts, c, pages.top_k, index), _workspace(workspace, index))
    return sel, sel_counts


def paged_decode_selected(cache: KVCache, layer_id: int, pages: SparsePages, q: torch.Tensor,
                          sel: torch.Tensor, sel_counts: torch.Tensor,
                          o: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                          stream=None) -> torch.Tensor:
    """paged_decode over the positions of the selected pages only; q, o:
    [batch, n_heads, head_dim], sel and sel_counts as select_pages gives them."""
    pg = pages.c_struct(cache)
    c, index = _cache(cache, pages.req_to_page, pg.req_to_page, 0, 0, True)
    dtype, heads = cache.k_buffer.dtype, _heads(q)
    if o is None:
        o = _empty(q.shape, q.dtype, cache.k_buffer.device, stream)
    scale = 1.0 / math.sqrt(c.head_dim) if sm_scale is None else float(sm_scale)
    _call("pkv_paged_decode_selected", index, stream, ctypes.byref(c), layer_id, ctypes.byref(pg),
            *_lists(sel, sel_counts, c, pages.top_k, index),
            _rows(q, "q", c, dtype, index, c.batch, heads), _rows(o, "o", c, dtype, index, c.batch, heads),
            heads, scale)
    return o


def sparse_decode_step(cache: KVCache, layer_id: int, pages: SparsePages, k_new: torch.Tensor,
                       v_new: torch.Tensor, q: torch.Tensor, o: Optional[torch.Tensor] = None,
                       sel: Optional[torch.Tensor] = None, sel_counts: Optional[torch.Tensor] = None,
                       sm_scale: Optional[float] = None, workspace: Optional[Workspace] = None,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """kv_write of k_new / v_new at cache.out_cache_loc, page_bounds,
    select_pages and paged_decode_selected as one call: (o, sel, sel_counts)."""
    n_new, heads, dtype = k_new.shape[0], _heads(q), cache.k_buffer.dtype
    pg = pages.c_struct(cache)
    c, index = _cache(cache, pages.req_to_page, pg.req_to_page, 0, n_new, True)
    if o is None:
        o = _empty(q.shape, q.dtype, cache.k_buffer.device, stream)
    if sel is None:
        sel = _empty((c.batch, c.n_kv_heads, pages.top_k), torch.int32, cache.k_buffer.device, stream)
    if sel_counts is None:
        sel_counts = _empty((c.batch, c.n_kv_heads), torch.int32, cache.k_buffer.device, stream)
    scale = 1.0 / math.sqrt(c.head_dim) if sm_scale is None else float(sm_scale)
    _call("pkv_sparse_decode_step", index, stream, ctypes.byref(c), layer_id, ctypes.byref(pg),
            _rows(k_new, "k_new", c, dtype, index, n_new, c.n_kv_heads),
            _rows(v_new, "v_new", c, dtype, index, n_new, c.n_kv_heads), n_new,
            _rows(q, "q", c, dtype, index, c.batch, heads), _rows(o, "o", c, dtype, index, c.batch, heads),
            heads, scale, *_lists(sel, sel_counts, c, pages.top_k, index), _workspace(workspace, index))
    return o, sel, sel_counts
