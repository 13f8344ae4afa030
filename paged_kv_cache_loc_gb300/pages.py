"""Python binding of the life of a cache's pages (include/pkv.h: pkv_copy_pages,
pkv_fork_requests, pkv_release_pages, pkv_compact_pages) and of the attention of
new tokens through the page table (pkv_paged_chunk).

Argument marshalling only, like sparse.py.  `shares` counts, for each page, the
references beyond the first: zeros to begin with, also for pages that
build_tables takes.  `free_pages`, `free_start` and `free_end` are build_tables'
list: the calls take from it or give back to it, and free_end[0] becomes its new
place.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional

import torch

from . import _lib
from ._lib import PkvKVCache, PkvPageState
from .ops import KVCache, Workspace, _DTYPES
from . import sparse
from .sparse import _call, _f32, _heads, _i32, _int32, _ints, _output, _pack_cache, _ptr, _rows, _st, _vp

_pack_state = struct.Struct("PiiPPPPiPP")
assert _pack_state.size == ctypes.sizeof(PkvPageState)
sparse._ARGS.update({
    "pkv_copy_pages": [_st, _i32, _vp, _vp, _vp, _i32, _vp],
    "pkv_fork_requests": [_st, _st, _vp, _vp],
    "pkv_release_pages": [_st, _st, _vp, _vp],
    "pkv_compact_pages": [_st, _st, _vp, _vp, _vp, _vp],
    "pkv_paged_chunk": [_st, _i32, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp],
})


def _describe(cache: KVCache, num_reqs: int, max_ctx_len: int, index: int, batched: bool, chunk: bool = False) -> bytes:
    """The packed descriptor of a cache's pool and, where `batched`, of its
    entries (request rows and lengths; with `chunk`, the places of their rows)."""
    kb, vb = cache.k_buffer, cache.v_buffer
    dtype, shape = kb.dtype, kb.shape
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported storage dtype {dtype}")
    if len(shape) != 4 or vb.shape != shape:
        raise ValueError("k_buffer/v_buffer must both be [n_layers, size, n_kv_heads, head_dim]")
    batch = rows = lens = qo = 0
    if batched:
        batch = cache.req_pool_indices.numel()
        if cache.seq_lens is None:
            raise ValueError("seq_lens is needed")
        rows, lens = _ptr(cache.req_pool_indices, "req_pool_indices", _int32, index), _ints(cache.seq_lens, "seq_lens", index, batch)
    if chunk:
        if cache.qo_indptr is None:
            raise ValueError("qo_indptr is needed")
        qo = _ints(cache.qo_indptr, "qo_indptr", index, batch + 1)
    return _pack_cache.pack(_ptr(kb, "k_buffer", dtype, index), _ptr(vb, "v_buffer", dtype, index), code, shape[0], shape[2],
                            shape[3], shape[1], 0, num_reqs, max_ctx_len, rows, lens, 0, qo, 0, batch, cache.max_len)


def _index(cache: KVCache) -> int:
    index = cache.k_buffer.get_device()
    if index < 0:
        raise ValueError("k_buffer must be a CUDA tensor (there is no CPU path)")
    return index


def _pages(cache: KVCache, page_size: int) -> int:
    if page_size < 1:
        raise ValueError("page_size must be positive")
    return cache.k_buffer.shape[1] // page_size


def _bounds(t: Optional[torch.Tensor], cache: KVCache, n_pages: int, index: int) -> int:
    if t is None:
        return 0
    n_layers, _, n_kv_heads, head_dim = cache.k_buffer.shape
    if t.shape != (n_layers, n_pages, n_kv_heads, 2, head_dim):
        raise ValueError("page_bounds must be [n_layers, size // page_size, n_kv_heads, 2, head_dim]")
    return _ptr(t, "page_bounds", cache.k_buffer.dtype, index)


def _state(cache: KVCache, req_to_page: torch.Tensor, page_size: int, shares: torch.Tensor, free_pages: torch.Tensor,
           free_start: torch.Tensor, free_end: Optional[torch.Tensor], page_bounds: Optional[torch.Tensor],
           token_table: bool, index: int) -> bytes:
    """The packed pkv_page_state."""
    if req_to_page.dim() != 2:
        raise ValueError("req_to_page must be [num_reqs, max_pages]")
    tokens = 0
    if token_table:
        table = cache.req_to_token
        if table.dim() != 2 or table.shape[0] != req_to_page.shape[0]:
            raise ValueError("req_to_token must be [num_reqs, max_ctx_len] with req_to_page's rows")
        tokens = _ptr(table, "req_to_token", _int32, index)
    n_pages = _pages(cache, page_size)
    return _pack_state.pack(
        _ptr(req_to_page, "req_to_page", _int32, index), req_to_page.shape[1], page_size, _ints(shares, "shares", index, n_pages),
        _ptr(free_pages, "free_pages", _int32, index), _ints(free_start, "free_start", index, 1),
        _ints(free_end, "free_end", index, 1), free_pages.numel(), tokens, _bounds(page_bounds, cache, n_pages, index))


def _table_len(cache: KVCache, token_table: bool) -> int:
    return cache.req_to_token.shape[1] if token_table and cache.req_to_token.dim() == 2 else 0


def copy_pages(cache: KVCache, page_size: int, src: torch.Tensor, dst: torch.Tensor,
               page_bounds: Optional[torch.Tensor] = None, stream=None) -> None:
    """Page dst[i] becomes a copy of page src[i] in every layer's K and V, and in
    page_bounds where given; pairs whose src is -1 are passed over."""
    index = _index(cache)
    n = src.numel()
    _call("pkv_copy_pages", index, stream, _describe(cache, 0, 0, index, False), page_size,
          _bounds(page_bounds, cache, _pages(cache, page_size), index), _ptr(src, "src", _int32, index), _ints(dst, "dst", index, n), n)


def fork_requests(cache: KVCache, req_to_page: torch.Tensor, page_size: int, parents: torch.Tensor, shares: torch.Tensor,
                  free_pages: torch.Tensor, free_start: torch.Tensor, free_end: torch.Tensor,
                  page_bounds: Optional[torch.Tensor] = None, token_table: bool = True, stream=None) -> None:
    """The rows cache.req_pool_indices take over the first cache.seq_lens
    positions of the rows `parents`: full pages are shared (shares + 1), a partly
    filled last page is copied to a page of the free list.  req_to_page follows,
    and cache.req_to_token unless token_table is False."""
    index = _index(cache)
    c = _describe(cache, req_to_page.shape[0], _table_len(cache, token_table), index, True)
    t = _state(cache, req_to_page, page_size, shares, free_pages, free_start, free_end, page_bounds, token_table, index)
    _call("pkv_fork_requests", index, stream, c, t, _ints(parents, "parents", index, cache.req_pool_indices.numel()))


def release_pages(cache: KVCache, req_to_page: torch.Tensor, page_size: int, shares: torch.Tensor, free_pages: torch.Tensor,
                  free_start: torch.Tensor, free_end: torch.Tensor, keep_lens: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """The rows cache.req_pool_indices, of cache.seq_lens positions, give up the
    pages behind their first keep_lens positions (None: all pages).  Pages that
    no row holds any more are written in front of the free list's place, in
    ascending order, and free_end[0] becomes the new place."""
    index = _index(cache)
    c = _describe(cache, req_to_page.shape[0], 0, index, True)
    t = _state(cache, req_to_page, page_size, shares, free_pages, free_start, free_end, None, False, index)
    _call("pkv_release_pages", index, stream, c, t, _ints(keep_lens, "keep_lens", index, cache.req_pool_indices.numel()))


def compact_workspace(n_pages: int, device="cuda") -> Workspace:
    """A workspace for compact_pages on a pool of n_pages pages."""
    need = _lib.load().pkv_compact_workspace_bytes(n_pages)
    if need == 0:
        raise ValueError("n_pages must be positive")
    return Workspace(1, 1, 64, -(-need // 256), device=device)      # 256 bytes of partials per split


def compact_pages(cache: KVCache, req_to_page: torch.Tensor, page_size: int, shares: torch.Tensor, free_pages: torch.Tensor,
                  free_start: torch.Tensor, remap: Optional[torch.Tensor] = None, free_out: Optional[torch.Tensor] = None,
                  page_bounds: Optional[torch.Tensor] = None, token_table: bool = True,
                  workspace: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """The used pages (those not in free_pages[free_start[0]:]) behind the pool's
    first U move to the free pages among them, U being their number.  shares,
    page_bounds, req_to_page and (unless token_table is False) cache.req_to_token
    follow; the list becomes U, U + 1, ... in free_out (None: in free_pages
    itself).  Returns remap, int32 [n_pages]: where each page went."""
    index = _index(cache)
    n_pages = _pages(cache, page_size)
    if free_out is None:
        free_out = free_pages
    c = _describe(cache, req_to_page.shape[0], _table_len(cache, token_table), index, False)
    t = _state(cache, req_to_page, page_size, shares, free_pages, free_start, None, page_bounds, token_table, index)
    if remap is None:
        remap = sparse._empty((n_pages,), _int32, cache.k_buffer.device, stream)
    _call("pkv_compact_pages", index, stream, c, t, _ints(free_out, "free_out", index, free_pages.numel()),
          _ints(remap, "remap", index, n_pages), sparse._workspace(workspace, index))
    return remap


def chunk_workspace_bytes(cache: KVCache, n_rows: int, n_heads: int, max_q_len: int) -> int:
    """Workspace bytes of a paged_chunk call of cache's batch and max_len with
    n_rows query rows, max_q_len for an entry at most."""
    index = _index(cache)
    c = PkvKVCache.from_buffer_copy(_describe(cache, 0, 0, index, True))
    with torch.cuda.device(index):
        return _lib.load().pkv_chunk_workspace_bytes(ctypes.byref(c), n_rows, n_heads, max_q_len)


def chunk_workspace(cache: KVCache, n_rows: int, n_heads: int, max_q_len: int) -> Workspace:
    """A workspace for paged_chunk calls of these sizes.  Other calls cut their
    contexts into the pieces that fit, or not at all: the same result, later."""
    need = chunk_workspace_bytes(cache, n_rows, n_heads, max_q_len)
    if need == 0:
        raise ValueError("sizes that paged_chunk refuses")
    return Workspace(1, 1, 64, -(-need // 256), device=cache.k_buffer.device)      # 256 bytes of partials per split


def paged_chunk(cache: KVCache, layer_id: int, req_to_page: torch.Tensor, page_size: int, q: torch.Tensor, max_q_len: int,
                causal: bool = True, o: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                workspace: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """Attention of each entry's rows cache.qo_indptr[b] .. cache.qo_indptr[b + 1]
    of q [n_q, n_heads, head_dim] (max_q_len at most) over its context of
    cache.seq_lens[b] positions (cache.max_len at most) through the page table:
    causal (the rows are the context's last tokens) or over all of it.  Rows that
    see nothing give 0."""
    if req_to_page.dim() != 2:
        raise ValueError("req_to_page must be [num_reqs, max_pages]")
    index = _index(cache)
    c = _describe(cache, req_to_page.shape[0], 0, index, True, chunk=True)
    heads, n_q, head_dim, dtype = _heads(q), q.shape[0], cache.k_buffer.shape[3], cache.k_buffer.dtype
    qp = _rows(q, "q", dtype, index, n_q, heads, head_dim)
    o, op = _output(o, q, dtype, index, stream)
    _call("pkv_paged_chunk", index, stream, c, layer_id, _ptr(req_to_page, "req_to_page", _int32, index), req_to_page.shape[1],
          page_size, qp, op, n_q, heads, max_q_len, 1 if causal else 0,
          1.0 / math.sqrt(head_dim) if sm_scale is None else sm_scale, sparse._workspace(workspace, index))
    return o
