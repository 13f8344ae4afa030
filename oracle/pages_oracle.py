"""CPU oracle of the life of a cache's pages (include/pkv.h: pkv_copy_pages,
pkv_fork_requests, pkv_release_pages, pkv_compact_pages): page by page, on numpy
arrays, sharing no code with the CUDA path.  K and V: [n_layers, size, ...];
bounds: [n_layers, n_pages, ...] or None.  Every function returns new arrays.
"""
import numpy as np


def _page(x, p, ps):
    return x[:, p * ps:(p + 1) * ps]


def copy_pages(k, v, bounds, ps, src, dst):
    k, v, bounds = k.copy(), v.copy(), None if bounds is None else bounds.copy()
    n_pages = k.shape[1] // ps
    for s, d in zip(src, dst):
        if s == -1 or s == d or not (0 <= s < n_pages and 0 <= d < n_pages):
            continue
        for x in (k, v):
            _page(x, d, ps)[...] = _page(x, s, ps)
        if bounds is not None:
            bounds[:, d] = bounds[:, s]
    return k, v, bounds


def fork(k, v, bounds, ps, table, tokens, shares, children, parents, lens, free, start):
    """(k, v, bounds, table, tokens, shares, free_end)."""
    k, v, bounds = k.copy(), v.copy(), None if bounds is None else bounds.copy()
    table, shares, tokens = table.copy(), shares.copy(), None if tokens is None else tokens.copy()
    for child, parent, n in zip(children, parents, lens):
        for i in range(n // ps):
            table[child, i] = table[parent, i]
            shares[table[parent, i]] += 1
        rest = n % ps
        if rest:
            i = n // ps
            new, old = free[start], table[parent, i]
            start += 1
            table[child, i] = new
            for x in (k, v):
                _page(x, new, ps)[:, :rest] = _page(x, old, ps)[:, :rest]
            if bounds is not None:
                bounds[:, new] = bounds[:, old]
        if tokens is not None:
            for j in range(n):
                tokens[child, j] = table[child, j // ps] * ps + j % ps
    return k, v, bounds, table, tokens, shares, start


def release(table, shares, ps, rows, lens, keep, free, start):
    """(table, shares, free, free_end)."""
    table, shares, free = table.copy(), shares.copy(), free.copy()
    gone = []
    for r, n, q in zip(rows, lens, keep):
        for i in range(-(-q // ps), -(-n // ps)):
            page = table[r, i]
            table[r, i] = -1
            if shares[page] == 0:
                gone.append(page)
            else:
                shares[page] -= 1
    free[start - len(gone):start] = np.sort(np.array(gone, free.dtype))
    return table, shares, free, start - len(gone)


def compact(k, v, bounds, ps, table, tokens, shares, free, start):
    """(k, v, bounds, table, tokens, shares, free, remap)."""
    n_pages = k.shape[1] // ps
    listed = set(int(p) for p in free[start:])
    used = [p for p in range(n_pages) if p not in listed]
    src = [p for p in used if p >= len(used)]
    dst = [p for p in range(len(used)) if p in listed]
    k, v, bounds = copy_pages(k, v, bounds, ps, src, dst)
    remap = np.arange(n_pages)
    shares, free = shares.copy(), free.copy()
    for s, d in zip(src, dst):
        remap[s] = d
        shares[d], shares[s] = shares[s], 0
    free[start:start + n_pages - len(used)] = np.arange(len(used), n_pages)
    table = table.copy()
    for i in np.ndindex(table.shape):
        if 0 <= table[i] < n_pages:
            table[i] = remap[table[i]]
    if tokens is not None:
        tokens = tokens.copy()
        for i in np.ndindex(tokens.shape):
            if 0 <= tokens[i] < n_pages * ps:
                tokens[i] = remap[tokens[i] // ps] * ps + tokens[i] % ps
    return k, v, bounds, table, tokens, shares, free, remap


def chunk(k, v, table, ps, rows, lens, qo_indptr, q, causal, scale, o):
    """Chunk attention in 64 bits over one layer's K and V [size, kv, d]; q [n_q,
    heads, d].  Returns (o with the entries' rows replaced, the largest sum_c
    |q_c k_c| |scale| of a pair that is seen, the largest |v| that is seen)."""
    k, v, q, o = (np.asarray(x, np.float64) for x in (k, v, q, o))
    o = o.copy()
    kv, g = k.shape[1], q.shape[1] // k.shape[1]
    most, largest = 0.0, 0.0
    for b, (r, n) in enumerate(zip(rows, lens)):
        lo, hi = qo_indptr[b], qo_indptr[b + 1]
        pos = np.arange(n)
        slots = table[r, pos // ps].astype(np.int64) * ps + pos % ps
        for i in range(lo, hi):
            m = n - (hi - lo) + (i - lo) + 1 if causal else n
            if m <= 0:
                o[i] = 0
                continue
            for h in range(kv):
                kk, vv, qq = k[slots[:m], h], v[slots[:m], h], q[i, h * g:(h + 1) * g]
                s = qq @ kk.T * scale
                w = np.exp(s - s.max(-1, keepdims=True))
                o[i, h * g:(h + 1) * g] = (w / w.sum(-1, keepdims=True)) @ vv
                most = max(most, (np.abs(qq) @ np.abs(kk).T).max() * abs(scale))
                largest = max(largest, np.abs(vv).max())
    return o, most, largest
