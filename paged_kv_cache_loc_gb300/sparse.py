"""Python binding of the sparse decode path and of the tables it reads
(include/pkv.h: pkv_build_tables, pkv_page_bounds, pkv_select_pages,
pkv_paged_decode_selected, pkv_sparse_decode_step).

Argument marshalling only, like ops.py.  These calls run once per layer and
step, and their kernels take less time than a few dozen Python calls, so a
tensor is checked by plain comparisons and a descriptor is packed in one call.
They work on the device of the cache, whatever the current one is; outputs that
are not given are allocated for the stream that the kernels run on.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import struct
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import PkvKVCache, PkvPages, PkvTables, check
from .ops import KVCache, Workspace, _DTYPES, _need

# The descriptors as bytes, field by field as in _lib (native sizes and alignment, padding at the end included).
_pack_cache = struct.Struct("PPiiiiqPiiPPPPPii")
_pack_pages = struct.Struct("PPiiiii0P")
_pack_tables = struct.Struct("PPiiPPPiiPPPPP")
for _s, _c in ((_pack_cache, PkvKVCache), (_pack_pages, PkvPages), (_pack_tables, PkvTables)):
    assert _s.size == ctypes.sizeof(_c)
_i32, _f32 = ctypes.c_int32, ctypes.c_float
_Tensor, _int32, _byref, _device = torch.Tensor, torch.int32, ctypes.byref, torch.cuda.current_device
_vp, _st = ctypes.c_void_p, ctypes.c_char_p                 # _st: a packed descriptor
# name -> argtypes, with the descriptors as bytes
_ARGS = {
    "pkv_build_tables": [_st, _st, _vp],
    "pkv_page_bounds": [_st, _i32, _st, _i32, _vp],
    "pkv_select_pages": [_st, _i32, _st, _vp, _i32, _vp, _vp, _vp, _vp],
    "pkv_paged_decode_selected": [_st, _i32, _st, _vp, _vp, _vp, _vp, _i32, _f32, _vp],
    "pkv_sparse_decode_step": [_st, _i32, _st, _vp, _vp, _i32, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _vp],
}
_functions = {}


def _function(name: str):
    """The library's function, loaded at its first call."""
    fn = _functions.get(name)
    if fn is None:
        fn = _lib.load()[name]              # an object of its own beside the library's attribute
        fn.restype, fn.argtypes = ctypes.c_int, _ARGS[name]
        _functions[name] = fn
    return fn


def _ptr(t: torch.Tensor, name: str, dtype, index: int) -> int:
    """The address of a contiguous tensor of `dtype` on CUDA device `index`,
    or in pinned host memory (as in ops._need)."""
    if type(t) is _Tensor and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return _need(t, name, dtype, torch.device("cuda", index))


def _ints(t: Optional[torch.Tensor], name: str, index: int, n: int) -> int:
    """The address of an int32 array of n elements; 0 for None."""
    if t is None:
        return 0
    p = _ptr(t, name, _int32, index)
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


def _describe(cache: KVCache, table: torch.Tensor, max_ctx_len: int, n_new: int, decode: bool):
    """The packed descriptor of a cache whose request rows are those of
    `table`: (bytes, address of the table, device index, storage dtype, shape of
    the pool, batch)."""
    kb, vb, rows, lens = cache.k_buffer, cache.v_buffer, cache.req_pool_indices, cache.seq_lens
    dtype, shape, index = kb.dtype, kb.shape, kb.get_device()
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported storage dtype {dtype}")
    if len(shape) != 4 or vb.shape != shape:
        raise ValueError("k_buffer/v_buffer must both be [n_layers, size, n_kv_heads, head_dim]")
    if index < 0:
        raise ValueError("k_buffer must be a CUDA tensor (there is no CPU path)")
    if table.dim() != 2:
        raise ValueError("req_to_page must be [num_reqs, max_pages]")
    if lens is None and decode:
        raise ValueError("seq_lens is needed")
    batch = rows.numel()
    loc = 0
    if n_new:
        loc = _ptr(cache.out_cache_loc, "out_cache_loc", _int32, index)
        if cache.out_cache_loc.numel() < n_new:     # it may be longer than what is written
            raise ValueError(f"out_cache_loc must have {n_new} elements at least, got {cache.out_cache_loc.numel()}")
    n_layers, size, n_kv_heads, head_dim = shape
    at = _ptr(table, "req_to_page", _int32, index)
    c = _pack_cache.pack(
        _ptr(kb, "k_buffer", dtype, index), _ptr(vb, "v_buffer", dtype, index), code, n_layers, n_kv_heads,
        head_dim, size, at, table.shape[0], max_ctx_len, _ptr(rows, "req_pool_indices", _int32, index),
        _ints(lens, "seq_lens", index, batch), 0, 0, loc, batch, cache.max_len)
    return c, at, index, dtype, shape, batch


def _describe_pages(pages: SparsePages, at: int, index: int, dtype, shape) -> bytes:
    """The packed descriptor of pages whose table is at `at`."""
    bounds, ps = pages.page_bounds, pages.page_size
    if ps < 1:
        raise ValueError("page_size must be positive")
    if bounds is None:
        p = 0
    else:
        n_layers, size, n_kv_heads, head_dim = shape
        if bounds.shape != (n_layers, size // ps, n_kv_heads, 2, head_dim):
            raise ValueError("page_bounds must be [n_layers, size // page_size, n_kv_heads, 2, head_dim]")
        p = _ptr(bounds, "page_bounds", dtype, index)
    return _pack_pages.pack(p, at, pages.req_to_page.shape[1], ps, pages.top_k, pages.n_first, pages.n_last)


def _rows(t: torch.Tensor, name: str, dtype, index: int, n: int, heads: int, head_dim: int) -> int:
    """The address of [n, heads, head_dim] rows."""
    if t.shape != (n, heads, head_dim):
        raise ValueError(f"{name} must be [{n}, {heads}, {head_dim}], got {list(t.shape)}")
    return _ptr(t, name, dtype, index)


def _outputs(sel: Optional[torch.Tensor], counts: Optional[torch.Tensor], batch: int, kv: int, top_k: int, device,
             index: int, stream):
    """sel and sel_counts, allocated where they are not given, and their addresses."""
    if sel is None:
        sel = _empty((batch, kv, top_k), _int32, device, stream)
        p = sel.data_ptr()
    else:
        p = _ints(sel, "sel", index, batch * kv * top_k)
    if counts is None:
        counts = _empty((batch, kv), _int32, device, stream)
        return sel, counts, p, counts.data_ptr()
    return sel, counts, p, _ints(counts, "sel_counts", index, batch * kv)


def _output(o: Optional[torch.Tensor], q: torch.Tensor, dtype, index: int, stream):
    """o, allocated like q where it is not given, and its address."""
    if o is None:
        o = _empty_like(q, stream) if q.is_cuda else _empty(q.shape, dtype, torch.device("cuda", index), stream)
        return o, o.data_ptr()
    if o.shape != q.shape:
        raise ValueError(f"o must be {list(q.shape)}, got {list(o.shape)}")
    return o, _ptr(o, "o", dtype, index)


def _heads(q: torch.Tensor) -> int:
    if q.dim() != 3:
        raise ValueError(f"q must be [batch, n_heads, head_dim], got {list(q.shape)}")
    return q.shape[1]


def _workspace(ws: Optional[Workspace], index: int):
    if ws is None:
        return None
    if ws.buffer.get_device() != index:
        raise ValueError(f"workspace is on {ws.buffer.device}, expected cuda:{index}")
    return _byref(ws.desc)


# the handle of a device's current stream, without the object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, index: int, stream, *args) -> None:
    """Calls the library's `name` on the cache's device with the stream's
    handle; None is the device's current stream."""
    fn = _functions.get(name) or _function(name)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if _device() == index:
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


def _empty_like(q: torch.Tensor, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty_like(q)
    with torch.cuda.stream(stream):
        return torch.empty_like(q)


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
    beyond out_cache_loc's length are an error on the device (they get no slot,
    but their pages are taken and entered in req_to_page); entries of
    out_cache_loc behind the last new token stay as they are."""
    tokens, loc = cache.req_to_token, cache.out_cache_loc
    if tokens.dim() != 2:
        raise ValueError("req_to_token must be [num_reqs, max_ctx_len]")
    n_new = 0 if loc is None else loc.numel()
    c, at, index, _, _, batch = _describe(cache, req_to_page, tokens.shape[1], n_new, True)
    if token_table and tokens.shape[0] != req_to_page.shape[0]:
        raise ValueError("req_to_page and req_to_token must have the same rows")
    t = _pack_tables.pack(
        _ints(q_lens, "q_lens", index, batch), at, req_to_page.shape[1], page_size,
        _ptr(free_pages, "free_pages", _int32, index), _ints(free_start, "free_start", index, 1),
        _ints(free_end, "free_end", index, 1), free_pages.numel(), n_new,
        _ints(cache.kv_indptr, "kv_indptr", index, batch + 1), _ints(cache.qo_indptr, "qo_indptr", index, batch + 1),
        _ints(positions, "positions", index, n_new), loc.data_ptr() if n_new else 0,
        _ptr(tokens, "req_to_token", _int32, index) if token_table else 0)
    _call("pkv_build_tables", index, stream, c, t)


def page_bounds(cache: KVCache, layer_id: int, pages: SparsePages, n_new: Optional[int] = None,
                stream=None) -> None:
    """Bring pages.page_bounds up to date with the keys written to the slots
    cache.out_cache_loc[:n_new] (None: all of them) of the layer."""
    if cache.out_cache_loc is None or pages.page_bounds is None:
        raise ValueError("out_cache_loc and page_bounds are needed")
    if n_new is None:
        n_new = cache.out_cache_loc.numel()
    c, at, index, dtype, shape, _ = _describe(cache, pages.req_to_page, 0, n_new, False)
    _call("pkv_page_bounds", index, stream, c, layer_id, _describe_pages(pages, at, index, dtype, shape), n_new)


def select_workspace_bytes(batch: int, n_kv_heads: int, max_len: int, page_size: int) -> int:
    """Workspace bytes that select_pages and sparse_decode_step need."""
    return _lib.load().pkv_select_workspace_bytes(batch, n_kv_heads, max_len, page_size)


def select_workspace(max_batch: int, n_kv_heads: int, max_len: int, page_size: int, device="cuda") -> Workspace:
    """A workspace for select_pages and sparse_decode_step of these sizes."""
    need = select_workspace_bytes(max_batch, n_kv_heads, max_len, page_size)
    if need == 0:
        raise ValueError("workspace dimensions must be positive")
    return Workspace(1, 1, 64, -(-need // 256), device=device)      # 256 bytes of partials per split


def select_pages(cache: KVCache, layer_id: int, pages: SparsePages, q: torch.Tensor,
                 sel: Optional[torch.Tensor] = None, sel_counts: Optional[torch.Tensor] = None,
                 workspace: Optional[Workspace] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The pages that each query of q [batch, n_heads, head_dim] attends to:
    sel int32 [batch, n_kv_heads, top_k] (logical pages, ascending, then -1)
    and sel_counts int32 [batch, n_kv_heads]."""
    c, at, index, dtype, shape, batch = _describe(cache, pages.req_to_page, 0, 0, True)
    heads, kv = _heads(q), shape[2]
    qp = _rows(q, "q", dtype, index, batch, heads, shape[3])
    sel, sel_counts, sp, cp = _outputs(sel, sel_counts, batch, kv, pages.top_k, cache.k_buffer.device, index, stream)
    _call("pkv_select_pages", index, stream, c, layer_id, _describe_pages(pages, at, index, dtype, shape), qp, heads, sp, cp,
          _workspace(workspace, index))
    return sel, sel_counts


def paged_decode_selected(cache: KVCache, layer_id: int, pages: SparsePages, q: torch.Tensor,
                          sel: torch.Tensor, sel_counts: torch.Tensor,
                          o: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                          stream=None) -> torch.Tensor:
    """paged_decode over the positions of the selected pages only; q, o:
    [batch, n_heads, head_dim], sel and sel_counts as select_pages gives them."""
    c, at, index, dtype, shape, batch = _describe(cache, pages.req_to_page, 0, 0, True)
    heads, kv, head_dim = _heads(q), shape[2], shape[3]
    qp = _rows(q, "q", dtype, index, batch, heads, head_dim)
    o, op = _output(o, q, dtype, index, stream)
    _call("pkv_paged_decode_selected", index, stream, c, layer_id, _describe_pages(pages, at, index, dtype, shape),
          _ints(sel, "sel", index, batch * kv * pages.top_k), _ints(sel_counts, "sel_counts", index, batch * kv), qp, op,
          heads, 1.0 / math.sqrt(head_dim) if sm_scale is None else sm_scale)
    return o


def sparse_decode_step(cache: KVCache, layer_id: int, pages: SparsePages, k_new: torch.Tensor,
                       v_new: torch.Tensor, q: torch.Tensor, o: Optional[torch.Tensor] = None,
                       sel: Optional[torch.Tensor] = None, sel_counts: Optional[torch.Tensor] = None,
                       sm_scale: Optional[float] = None, workspace: Optional[Workspace] = None,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """kv_write of k_new / v_new at cache.out_cache_loc, page_bounds,
    select_pages and paged_decode_selected as one call: (o, sel, sel_counts)."""
    n_new, heads = k_new.shape[0], _heads(q)
    c, at, index, dtype, shape, batch = _describe(cache, pages.req_to_page, 0, n_new, True)
    kv, head_dim = shape[2], shape[3]
    qp = _rows(q, "q", dtype, index, batch, heads, head_dim)
    kp = _rows(k_new, "k_new", dtype, index, n_new, kv, head_dim)
    vp = _rows(v_new, "v_new", dtype, index, n_new, kv, head_dim)
    o, op = _output(o, q, dtype, index, stream)
    sel, sel_counts, sp, cp = _outputs(sel, sel_counts, batch, kv, pages.top_k, cache.k_buffer.device, index, stream)
    _call("pkv_sparse_decode_step", index, stream, c, layer_id, _describe_pages(pages, at, index, dtype, shape), kp, vp, n_new,
          qp, op, heads, 1.0 / math.sqrt(head_dim) if sm_scale is None else sm_scale, sp, cp, _workspace(workspace, index))
    return o, sel, sel_counts
