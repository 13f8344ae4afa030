// pkv_pages.cu -- the life of a cache's pages on the GPU: copies of pages
// (pkv_copy_pages), request rows that share or copy another row's pages
// (pkv_fork_requests), pages given back to the free list (pkv_release_pages),
// and the used pages moved to the pool's front (pkv_compact_pages).
//
// A page is, per layer, one run of page_size rows in k_buffer and one in
// v_buffer, and one run of 2 n_kv_heads head_dim elements in page_bounds, so
// every copy here is of long contiguous runs: consecutive threads take
// consecutive 16-byte chunks, several in flight per thread.
//
// shares[page] counts the references beyond the first, so the pages that
// pkv_build_tables takes from the free list need no entry of their own, and a
// reference that is dropped at 0 is the last one: the count then stands below
// 0, which marks the page as released until the end of the call.
#include <cooperative_groups.h>

#include "pkv_common.cuh"
#include "pkv_launch.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kThreads = 256;              // copying CTAs
constexpr int kUnroll = 8;                 // 16-byte chunks in flight per thread
constexpr int kPiece = kThreads * kUnroll;   // chunks per CTA and step: 32 KB
constexpr int kScanThreads = 1024;         // CTAs of the one cluster that scans the pool's pages
constexpr int kScanWarps = kScanThreads / 32;

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }
__device__ __forceinline__ bool in_range(long long x, long long n) {
    return static_cast<unsigned long long>(x) < static_cast<unsigned long long>(n);
}

// chunks [at, at + kPiece) of a run of n chunks
__device__ __forceinline__ void copy_piece(uint4 *dst, const uint4 *src, int64_t at, int64_t n) {
    uint4 v[kUnroll];
    const int64_t i0 = at + threadIdx.x;
    if (at + kPiece <= n) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = __ldcs(src + i0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) __stcs(dst + i0 + u * kThreads, v[u]);
    } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i0 + u * kThreads < n) v[u] = __ldcs(src + i0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i0 + u * kThreads < n) __stcs(dst + i0 + u * kThreads, v[u]);
    }
}

// Piece `unit` of the copy of one page: per layer the pieces of K, of V and of
// the bounds.
__device__ __forceinline__ void copy_page_unit(const PageRuns &r, int64_t src, int64_t dst, int64_t unit) {
    const int64_t layer = static_cast<uint32_t>(unit) / static_cast<uint32_t>(r.layer_units);
    int u = static_cast<int>(unit - layer * r.layer_units);
    const int64_t s = layer * r.n_pages + src, d = layer * r.n_pages + dst;
    if (u < 2 * r.page_units) {
        uint4 *buf = static_cast<uint4 *>(u < r.page_units ? r.k_buffer : r.v_buffer);
        if (u >= r.page_units) u -= r.page_units;
        copy_piece(buf + d * r.page_chunks, buf + s * r.page_chunks, static_cast<int64_t>(u) * kPiece, r.page_chunks);
    } else {
        uint4 *buf = static_cast<uint4 *>(r.page_bounds);
        u -= 2 * r.page_units;
        copy_piece(buf + d * r.bound_chunks, buf + s * r.bound_chunks, static_cast<int64_t>(u) * kPiece, r.bound_chunks);
    }
}

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyPagesParams p) {
    const int64_t per = static_cast<int64_t>(p.runs.n_layers) * p.runs.layer_units;
    for (int64_t i = blockIdx.x; i < p.n * per; i += gridDim.x) {
        const int64_t pair = i / per;
        const int src = __ldg(p.src + pair), dst = __ldg(p.dst + pair);
        if (src == -1 || src == dst) continue;
        if (!in_range(src, p.runs.n_pages) || !in_range(dst, p.runs.n_pages)) {
            if (threadIdx.x == 0) record_error(p.err, in_range(src, p.runs.n_pages) ? dst : src);
            continue;
        }
        copy_page_unit(p.runs, src, dst, i - pair * per);
    }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

struct ForkEntry {
    int child, parent, len;
    bool part;                 // takes a page of the free list
};

__device__ __forceinline__ ForkEntry load_fork(const ForkParams &p, int b, bool report) {
    ForkEntry e;
    e.child = __ldg(p.children + b);
    e.parent = __ldg(p.parents + b);
    e.len = __ldg(p.seq_lens + b);
    bool ok = true;
    int bad = 0;
    if (!in_range(e.child, p.num_reqs)) ok = false, bad = e.child;
    else if (!in_range(e.parent, p.num_reqs)) ok = false, bad = e.parent;
    else if (!in_range(e.len, static_cast<long long>(p.max_len) + 1)) ok = false, bad = e.len;
    else if (e.child == e.parent && e.len > 0) ok = false, bad = e.child;
    if (!ok) {
        if (report) record_error(p.err, bad);
        e.len = 0;
    }
    e.part = e.len % p.page_size != 0;
    return e;
}

// One CTA per (slice, entry).  Every CTA finds the entry's place in the free
// list by itself, counting the entries before it that take a page (the lengths
// come from L2), so nothing passes between CTAs and one launch does it all; the
// first slice writes the table row and the counts, all of them share the
// token row and the copy of the partly filled page.
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ ForkParams p) {
    __shared__ int warp_count[kThreads / 32];
    const int b = blockIdx.y, slice = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const ForkEntry e = b < p.batch ? load_fork(p, b, slice == 0 && tid == 0) : ForkEntry{0, 0, 0, false};   // no entries: one CTA
    int before = 0;
    for (int i = tid; i < b; i += kThreads) before += load_fork(p, i, false).part;
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) warp_count[tid >> 5] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) before += warp_count[w];
    int start = __ldg(p.free_start);
    if (!in_range(start, static_cast<long long>(p.n_free) + 1)) {
        if (b == 0 && slice == 0 && tid == 0) record_error(p.err, start);
        start = p.n_free;
    }
    const long long place = static_cast<long long>(start) + before;
    const bool lead = slice == 0 && tid == 0;
    if (lead && b == max(p.batch, 1) - 1) *p.free_end = static_cast<int>(min(place + e.part, static_cast<long long>(p.n_free)));
    if (e.len == 0) return;

    const int ps = p.page_size, full = e.len / ps, rest = e.len - full * ps;
    const int32_t *theirs = p.req_to_page + static_cast<int64_t>(e.parent) * p.max_pages;
    int32_t *mine = p.req_to_page + static_cast<int64_t>(e.child) * p.max_pages;
    int fresh = -1, old = -1;
    if (e.part) {
        if (place >= p.n_free) {
            if (lead) record_error(p.err, -300000LL - b);
        } else {
            fresh = __ldg(p.free_pages + place);
            if (!in_range(fresh, p.n_pages)) {
                if (lead) record_error(p.err, fresh);
                fresh = -1;
            }
        }
        old = theirs[full];
        if (!in_range(old, p.n_pages)) {
            if (lead) record_error(p.err, old);
            old = -1;
        }
        if (lead) mine[full] = fresh;
    }
    // (unsigned: a row may hold 2^31 - 1 positions, and the last step goes beyond)
    for (uint32_t i = slice * kThreads + tid; i < static_cast<uint32_t>(full); i += gridDim.x * kThreads) {
        int page = theirs[i];
        if (in_range(page, p.n_pages)) {
            atomicAdd(p.shares + page, 1);
        } else {
            record_error(p.err, page);
            page = -1;
        }
        mine[i] = page;
    }
    if (p.req_to_token) {
        int32_t *tokens = p.req_to_token + static_cast<int64_t>(e.child) * p.max_ctx_len;
        for (uint32_t j = slice * kThreads + tid; j < static_cast<uint32_t>(e.len); j += gridDim.x * kThreads) {
            const int i = j / ps;
            const int page = i < full ? theirs[i] : fresh;
            tokens[j] = in_range(page, p.n_pages) ? page * ps + (j - i * ps) : -1;
        }
    }
    if (fresh < 0 || old < 0 || fresh == old) return;
    // the first `rest` rows of the page in every layer's K and V, then the bounds
    const PageRuns &r = p.runs;
    // (counts that the host has found to fit 31 bits)
    const uint32_t bound = static_cast<uint32_t>(r.bound_chunks), run = rest * (static_cast<uint32_t>(r.page_chunks) / ps);
    const uint32_t rows = 2 * run * r.n_layers, total = rows + (r.page_bounds ? r.n_layers * bound : 0);
    for (uint32_t at = slice * kPiece; at < total; at += gridDim.x * kPiece) {
        uint4 v[kUnroll];
        uint4 *to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t i = at + tid + u * kThreads;
            to[u] = nullptr;
            if (i >= total) continue;
            uint4 *buf;
            int64_t s, d;
            if (i < rows) {
                const uint32_t half = i / run, off = i - half * run;
                const int64_t layer = half >> 1;
                buf = static_cast<uint4 *>(half & 1 ? r.v_buffer : r.k_buffer);
                s = (layer * r.n_pages + old) * r.page_chunks + off;
                d = (layer * r.n_pages + fresh) * r.page_chunks + off;
            } else {
                const int64_t layer = (i - rows) / bound, off = i - rows - layer * bound;
                buf = static_cast<uint4 *>(r.page_bounds);
                s = (layer * r.n_pages + old) * r.bound_chunks + off;
                d = (layer * r.n_pages + fresh) * r.bound_chunks + off;
            }
            v[u] = __ldcs(buf + s);
            to[u] = buf + d;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u]) __stcs(to[u], v[u]);
    }
}

// ---------------------------------------------------------------------------
// release
// ---------------------------------------------------------------------------

// The pages [lo, hi) of its row that entry b gives up.
struct ReleaseEntry {
    int row, lo, hi;
};

__device__ __forceinline__ ReleaseEntry load_release(const ReleaseParams &p, int b, bool report) {
    const int row = __ldg(p.req_pool_indices + b), len = __ldg(p.seq_lens + b);
    const int keep = p.keep_lens ? __ldg(p.keep_lens + b) : 0;
    bool ok = true;
    int bad = 0;
    if (!in_range(row, p.num_reqs)) ok = false, bad = row;
    else if (!in_range(len, static_cast<long long>(p.max_len) + 1)) ok = false, bad = len;
    else if (!in_range(keep, static_cast<long long>(len) + 1)) ok = false, bad = keep;
    if (!ok) {
        if (report) record_error(p.err, bad);
        return {0, 0, 0};
    }
    return {row, ceil_div(keep, p.page_size), ceil_div(len, p.page_size)};
}

// Column i of an entry's row is given up.  The exchange makes a row that is
// named twice give each page up once.
__device__ __forceinline__ void drop_page(const ReleaseParams &p, const ReleaseEntry &e, int i) {
    const int page = atomicExch(p.req_to_page + static_cast<int64_t>(e.row) * p.max_pages + i, -1);
    if (!in_range(page, p.n_pages)) {
        record_error(p.err, page);
        return;
    }
    atomicSub(p.shares + page, 1);
}

__global__ void __launch_bounds__(kThreads) drop_kernel(const __grid_constant__ ReleaseParams p) {
    const int b = blockIdx.y;
    const ReleaseEntry e = load_release(p, b, blockIdx.x == 0 && threadIdx.x == 0);
    // (unsigned: a row may hold 2^31 - 1 pages, and the last step goes beyond)
    for (uint32_t i = e.lo + blockIdx.x * kThreads + threadIdx.x; i < static_cast<uint32_t>(e.hi); i += gridDim.x * kThreads) drop_page(p, e, i);
}

// Exclusive sums of two counts of the warps over the cluster, in warp order, and
// their totals.  Ends with every CTA's counts read.
__device__ __forceinline__ void cluster_prefix(cg::cluster_group &cluster, int2 *counts, int2 mine, int2 *before, int2 *total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster.block_rank();
    if (lane == 0) counts[warp] = mine;
    cluster.sync();
    int2 pre = make_int2(0, 0), all = make_int2(0, 0);
    for (int r = 0; r < static_cast<int>(cluster.num_blocks()); ++r) {
        const int2 x = cluster.map_shared_rank(counts, r)[lane];
        const bool earlier = r < rank || (r == rank && lane < warp);
        pre.x += earlier ? x.x : 0;
        pre.y += earlier ? x.y : 0;
        all.x += x.x;
        all.y += x.y;
    }
    cluster.sync();
    *before = make_int2(__reduce_add_sync(0xffffffffu, pre.x), __reduce_add_sync(0xffffffffu, pre.y));
    *total = make_int2(__reduce_add_sync(0xffffffffu, all.x), __reduce_add_sync(0xffffffffu, all.y));
}

// Pages [lo, hi) of this warp of the cluster: whole 128-page blocks.
__device__ __forceinline__ void warp_range(int rank, int blocks, int64_t n_pages, int64_t *lo, int64_t *hi) {
    const int64_t warps = static_cast<int64_t>(blocks) * kScanWarps, w = static_cast<int64_t>(rank) * kScanWarps + (threadIdx.x >> 5);
    const int64_t per = ((n_pages + 127) / 128 + warps - 1) / warps * 128;
    *lo = min(n_pages, w * per);
    *hi = min(n_pages, *lo + per);
}

// Four counts of the pool's pages from page i on (16-byte aligned where i is a
// multiple of four); pages behind the end read as `none`.
__device__ __forceinline__ int4 load4(const int32_t *a, int64_t i, int64_t hi, int none, bool vec) {
    if (vec && i + 3 < hi) return __ldcg(reinterpret_cast<const int4 *>(a + i));
    int4 v = make_int4(none, none, none, none);
    if (i < hi) v.x = __ldcg(a + i);
    if (i + 1 < hi) v.y = __ldcg(a + i + 1);
    if (i + 2 < hi) v.z = __ldcg(a + i + 2);
    if (i + 3 < hi) v.w = __ldcg(a + i + 3);
    return v;
}

// One cluster: the released pages (counts below 0) in ascending order in front
// of the free list.  kDrop: the references are dropped here too, a warp per
// entry at a time.
template <bool kDrop>
__global__ void __launch_bounds__(kScanThreads) collect_kernel(const __grid_constant__ ReleaseParams p) {
    __shared__ int2 counts[kScanWarps];
    __shared__ int lists[kScanWarps][128];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), blocks = cluster.num_blocks(), lane = threadIdx.x & 31;
    if (kDrop) {
        for (int b = (threadIdx.x >> 5) * blocks + rank; b < p.batch; b += blocks * kScanWarps) {
            const ReleaseEntry e = load_release(p, b, lane == 0);
            for (int i = e.lo + lane; i < e.hi; i += 32) drop_page(p, e, i);
        }
        cluster.sync();
    } else {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
    }
    int start = __ldg(p.free_start);
    if (!in_range(start, static_cast<long long>(p.n_free) + 1)) {
        if (rank == 0 && threadIdx.x == 0) record_error(p.err, start);
        start = p.n_free;
    }
    int64_t lo, hi;
    warp_range(rank, blocks, p.n_pages, &lo, &hi);
    const bool vec = (reinterpret_cast<uintptr_t>(p.shares) & 15) == 0;
    // both passes load kBlocks blocks of 128 pages before they look at the first
    constexpr int kBlocks = 4;
    int4 v[kBlocks];
    auto load = [&](int64_t i0) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) v[k] = load4(p.shares, i0 + 128 * k + 4 * lane, hi, 0, vec);
    };
    int n = 0;
    for (int64_t i0 = lo; i0 < hi; i0 += 128 * kBlocks) {
        load(i0);
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int least = min(min(v[k].x, v[k].y), min(v[k].z, v[k].w));
            n += (v[k].x < 0) + (v[k].y < 0) + (v[k].z < 0) + (v[k].w < 0);
            if (least < -1)                              // more references dropped than there were
                record_error(p.err, -400000LL - (i0 + 128 * k + 4 * lane + (v[k].x < -1 ? 0 : v[k].y < -1 ? 1 : v[k].z < -1 ? 2 : 3)));
        }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    int2 sums_before, sums;
    cluster_prefix(cluster, counts, make_int2(n, 0), &sums_before, &sums);
    const int before = sums_before.x, total = sums.x;
    if (rank == 0 && threadIdx.x == 0) {
        if (total > start) record_error(p.err, total);
        *p.free_end = max(0, start - total);
    }
    if (n == 0) return;
    int at = start - total + before;
    int *list = lists[threadIdx.x >> 5];                 // a block's pages, so that they are stored side by side
    for (int64_t i0 = lo; i0 < hi; i0 += 128 * kBlocks) {
        load(i0);
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int c[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            const int mine = (c[0] < 0) + (c[1] < 0) + (c[2] < 0) + (c[3] < 0);
            if (!__any_sync(0xffffffffu, mine)) continue;
            int inc = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += y;
            }
            const int64_t i = i0 + 128 * k + 4 * lane;
            int to = inc - mine;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c[u] < 0) list[to++] = static_cast<int>(i + u);
            if (vec && i + 3 < hi) {
                if (mine) *reinterpret_cast<int4 *>(p.shares + i) = make_int4(max(c[0], 0), max(c[1], 0), max(c[2], 0), max(c[3], 0));
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c[u] < 0) p.shares[i + u] = 0;
            }
            __syncwarp();
            const int n_block = __shfl_sync(0xffffffffu, inc, 31);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int s = lane + 32 * u;
                if (s < n_block && at + s >= 0) p.free_pages[at + s] = list[s];
            }
            __syncwarp();
            at += n_block;
        }
    }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------

// One cluster: which page goes where.  remap serves as the marks first (-1 free,
// 0 used); moves[0] becomes the number of moves, then the places they go to and,
// from `cap` on, the pages they come from, each in ascending order.
__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int2 counts[kScanWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), blocks = cluster.num_blocks(), lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(rank) * kScanThreads + threadIdx.x, step = static_cast<int64_t>(blocks) * kScanThreads;
    const int64_t n = p.runs.n_pages;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    for (int64_t i = first; i < n; i += step) p.remap[i] = 0;
    cluster.sync();
    int start = __ldg(p.free_start);
    if (!in_range(start, static_cast<long long>(p.n_free) + 1)) {
        if (first == 0) record_error(p.err, start);
        start = p.n_free;
    }
    int mine = 0;
    for (int64_t i = start + first; i < p.n_free; i += step) {
        const int page = p.free_pages[i];
        if (!in_range(page, n) || atomicExch(p.remap + page, -1) == -1) record_error(p.err, page);
        else ++mine;
    }
    int2 before, sums;
    cluster_prefix(cluster, counts, make_int2(__reduce_add_sync(0xffffffffu, mine), 0), &before, &sums);
    const int n_free = sums.x;
    const int64_t used = n - n_free;
    int64_t lo, hi;
    warp_range(rank, blocks, n, &lo, &hi);
    const bool vec = (reinterpret_cast<uintptr_t>(p.remap) & 15) == 0;
    // The free pages before each warp's, and those among the first `used`: as many
    // used pages stand behind.  A hole's rank is the free pages before it, a used
    // page's behind the first `used` what is left of its place without them.
    auto marks = [&](int64_t i, int (&m)[4]) {
        const int4 v = load4(p.remap, i, hi, 0, vec);
        m[0] = v.x, m[1] = v.y, m[2] = v.z, m[3] = v.w;
    };
    int free = 0, holes = 0;
    for (int64_t i = lo + 4 * lane; i < hi; i += 128) {
        int m[4];
        marks(i, m);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            free += m[u] != 0;
            holes += m[u] != 0 && i + u < used;
        }
    }
    cluster_prefix(cluster, counts, make_int2(__reduce_add_sync(0xffffffffu, free), __reduce_add_sync(0xffffffffu, holes)), &before, &sums);
    int at = before.x;
    const int n_moves = sums.y;
    int32_t *to = p.moves + 4, *from = to + p.cap;
    for (int64_t i0 = lo; i0 < hi; i0 += 128) {
        const int64_t i = i0 + 4 * lane;
        int m[4];
        marks(i, m);
        const int c = (m[0] != 0) + (m[1] != 0) + (m[2] != 0) + (m[3] != 0);
        int inc = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        int before_me = at + inc - c;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i + u >= hi) break;
            if (i + u < used) {
                if (m[u]) to[before_me] = static_cast<int>(i + u);
            } else if (!m[u]) {
                from[i + u - used - (before_me - n_moves)] = static_cast<int>(i + u);
            }
            before_me += m[u] != 0;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
        if (vec && i + 3 < hi) {
            *reinterpret_cast<int4 *>(p.remap + i) = make_int4(static_cast<int>(i), static_cast<int>(i + 1), static_cast<int>(i + 2), static_cast<int>(i + 3));
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u < hi) p.remap[i + u] = static_cast<int>(i + u);
        }
    }
    cluster.sync();
    for (int64_t i = first; i < n_moves; i += step) {
        const int d = __ldcg(to + i), s = __ldcg(from + i);
        p.remap[s] = d;
        p.shares[d] = __ldcg(p.shares + s);
        p.shares[s] = 0;
    }
    // (fewer than listed after an error: behind them no page that may hold a row's by now)
    for (int64_t i = first; i < p.n_free - start; i += step) p.free_out[start + i] = i < n_free ? static_cast<int>(used + i) : -1;
    if (first == 0) p.moves[0] = n_moves;
}

// The moves' copies and the tables' new entries: every CTA takes a share of both.
__global__ void __launch_bounds__(kThreads) compact_move_kernel(const __grid_constant__ CompactParams p) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int64_t n = p.runs.n_pages;
    const int n_moves = __ldcg(p.moves);
    const int64_t per = static_cast<int64_t>(p.runs.n_layers) * p.runs.layer_units;
    for (int64_t i = blockIdx.x; i < n_moves * per; i += gridDim.x) {
        const int64_t m = i / per;
        copy_page_unit(p.runs, __ldcg(p.moves + 4 + p.cap + m), __ldcg(p.moves + 4 + m), i - m * per);
    }
    if (n_moves == 0) return;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = first; i < p.table_entries; i += step) {
        const int page = p.req_to_page[i];
        if (!in_range(page, n)) continue;
        const int to = __ldcg(p.remap + page);
        if (to != page) p.req_to_page[i] = to;
    }
    for (int64_t i = first; i < p.token_entries; i += step) {
        const int slot = p.req_to_token[i];
        const int page = slot / p.page_size;
        if (slot < 0 || page >= n) continue;
        const int to = __ldcg(p.remap + page);
        if (to != page) p.req_to_token[i] = to * p.page_size + (slot - page * p.page_size);
    }
}

// The launch of a single cluster of eight CTAs, or of a dependent grid.
template <typename P>
cudaError_t launch(void (*kernel)(P), const P &p, dim3 grid, int threads, int cluster, bool dependent, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

constexpr int kScanCluster = 8;

}  // namespace

void page_runs_units(PageRuns *r) {
    r->page_units = static_cast<int32_t>((r->page_chunks + kPiece - 1) / kPiece);
    const int bound_units = r->page_bounds ? static_cast<int32_t>((r->bound_chunks + kPiece - 1) / kPiece) : 0;
    r->layer_units = 2 * r->page_units + bound_units;
}

cudaError_t launch_copy_pages(const CopyPagesParams &p, cudaStream_t s) {
    // a CTA per piece of 32 KB, which the hardware hands out as others end (2.3 GB of pages
    // of 16: 337 us; 342 with eight CTAs per SM that go on to their next pieces.  Runs of
    // 2 KB, 1024 pages of one slot in 32 layers, 281 and 238)
    const int64_t units = p.n * p.runs.n_layers * p.runs.layer_units;
    const int64_t most = 1 << 20;
    copy_pages_kernel<<<static_cast<unsigned>(units < most ? units : most), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_fork(const ForkParams &p, int sms, cudaStream_t s) {
    // CTAs enough for eight on an SM, none with less than one step of a full page's copy.
    // Where a page is small and the parent long, the rows of the tables are then the work
    // of few CTAs (one child of 128K positions in pages of 16, one layer: 35 us, 6 with
    // CTAs by the row's length; 8 x 128K in pages of one 228 and 12; with a model's layers
    // it makes no difference: 256 children of 0.5K to 4K, 8 layers, 27 either way)
    const int64_t chunks = p.runs.n_layers * (2 * p.runs.page_chunks + (p.runs.page_bounds ? p.runs.bound_chunks : 0));
    int64_t slices = (chunks + kPiece - 1) / kPiece;
    const int batch = p.batch > 0 ? p.batch : 1;
    const int64_t most = (8LL * sms + batch - 1) / batch;
    if (slices > most) slices = most;
    if (slices < 1) slices = 1;
    fork_kernel<<<dim3(static_cast<unsigned>(slices), batch), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_release(const ReleaseParams &p, int sms, cudaStream_t s) {
    // Up to 64K table entries the cluster that collects the pages drops the references
    // too, a warp per row: one launch in place of two saves the host 2.3 us of 11.5 a
    // call.  The GPU takes longer by it, the more the longer the rows: 64 requests that
    // give up to 12 positions each 10.3 us against 9.6 in two launches, 64 x 255 pages 14.4
    // and 10.6, 512 x 127 17.4 and 11.4, one row of 4095 pages 59 and 10, of 65535 746 and 12.
    // Above, two launches are far ahead (512 rows of 0.1K to 2K pages 30 us, 87 in one).
    if (static_cast<int64_t>(p.batch) * p.max_pages <= 1 << 16)
        return launch(collect_kernel<true>, p, dim3(kScanCluster), kScanThreads, kScanCluster, false, s);
    int64_t x = (static_cast<int64_t>(p.max_pages) + kThreads - 1) / kThreads;
    const int64_t most = (16LL * sms + p.batch - 1) / p.batch;
    if (x > most) x = most;
    drop_kernel<<<dim3(static_cast<unsigned>(x), p.batch), kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch(collect_kernel<false>, p, dim3(kScanCluster), kScanThreads, kScanCluster, true, s);
}

cudaError_t launch_compact(const CompactParams &p, int sms, cudaStream_t s) {
    cudaError_t e = launch(compact_plan_kernel, p, dim3(kScanCluster), kScanThreads, kScanCluster, false, s);
    if (e != cudaSuccess) return e;
    return launch(compact_move_kernel, p, dim3(static_cast<unsigned>(8 * sms)), kThreads, 1, true, s);
}

}  // namespace pkv
