"""fp64 oracle of the sparse decode path and of the tables it reads.

TEST INFRASTRUCTURE ONLY (like the rest of this package): plain numpy, entry by
entry, from the definitions in include/pkv.h.  Keys, bounds and queries come
widened to float64; nothing here rounds.
"""
from __future__ import annotations

import numpy as np


def build_tables(rows, lens, q_lens, req_to_page, page_size, free_pages, free_start):
    """dict of kv_indptr, qo_indptr, positions, out_cache_loc, req_to_page and
    free_end; lengths are valid and the free list is long enough."""
    table = np.array(req_to_page, np.int64)
    take = int(free_start)
    loc, pos = [], []
    for r, n, q in zip(rows, lens, q_lens):
        for p in range(n - q, n):
            if p % page_size == 0:
                table[r, p // page_size] = free_pages[take]
                take += 1
            loc.append(table[r, p // page_size] * page_size + p % page_size)
            pos.append(p)
    return dict(kv_indptr=np.r_[0, np.cumsum(lens)].astype(np.int64), qo_indptr=np.r_[0, np.cumsum(q_lens)].astype(np.int64),
                positions=np.array(pos, np.int64), out_cache_loc=np.array(loc, np.int64), req_to_page=table, free_end=take)


def page_bounds(bounds, keys, loc, page_size):
    """bounds [n_pages, kv, 2, d] after the keys [n, kv, d] went to slots loc,
    one after the other."""
    b = np.array(bounds, np.float64)
    for k, slot in zip(np.asarray(keys, np.float64), loc):
        page, off = divmod(int(slot), page_size)
        if off == 0:
            b[page, :, 0] = b[page, :, 1] = k
        else:
            b[page, :, 0] = np.minimum(b[page, :, 0], k)      # numpy's minimum keeps a NaN
            b[page, :, 1] = np.maximum(b[page, :, 1], k)
    return b


def page_scores(bounds, pages, q, g):
    """Scores of physical pages for one kv head: q [G, d]."""
    with np.errstate(invalid="ignore", over="ignore"):
        lo, hi = bounds[pages, g, 0], bounds[pages, g, 1]
        most = np.where(q[:, None] >= 0, q[:, None] * hi, q[:, None] * lo).sum(-1)
        return most.max(0) if len(q) else most


def select_pages(bounds, req_to_page, rows, lens, q, page_size, top_k, n_first, n_last):
    """(sel [batch, kv, top_k], counts [batch, kv]); q [batch, heads, d]."""
    batch, heads, _ = q.shape
    kv = bounds.shape[1]
    sel, counts = np.full((batch, kv, top_k), -1, np.int64), np.zeros((batch, kv), np.int64)
    for b in range(batch):
        n = -(-int(lens[b]) // page_size)
        for g in range(kv):
            if n <= top_k:
                pick = np.arange(n)
            else:
                qg = q[b, g * (heads // kv):(g + 1) * (heads // kv)]
                s = page_scores(bounds, req_to_page[rows[b], :n], qg, g)
                forced = (np.arange(n) < n_first) | (np.arange(n) >= n - n_last)
                rank = np.where(np.isnan(s), np.inf, s)
                pick = np.sort(np.lexsort((np.arange(n), ~np.isnan(s), -rank, ~forced))[:top_k])
            sel[b, g, :len(pick)], counts[b, g] = pick, len(pick)
    return sel, counts


def decode_selected(k, v, req_to_page, rows, lens, sel, counts, q, page_size, sm_scale):
    """(o [batch, heads, d], the largest sum_c |q_c k_c| * sm_scale of a pair)
    over the listed pages; k, v [size, kv, d]."""
    batch, heads, d = q.shape
    kv = k.shape[1]
    o, reach = np.zeros((batch, heads, d)), 0.0
    for b in range(batch):
        for g in range(kv):
            slots = []
            for p in sel[b, g, :counts[b, g]]:
                n = min(page_size, int(lens[b]) - int(p) * page_size)
                slots.append(int(req_to_page[rows[b], p]) * page_size + np.arange(n))
            slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
            if not len(slots):
                continue
            for h in range(g * (heads // kv), (g + 1) * (heads // kv)):
                w = k[slots, g] @ q[b, h] * sm_scale
                reach = max(reach, float((np.abs(k[slots, g]) @ np.abs(q[b, h])).max()) * abs(sm_scale))
                w = np.exp(w - w.max())
                o[b, h] = w @ v[slots, g] / w.sum()
    return o, reach
