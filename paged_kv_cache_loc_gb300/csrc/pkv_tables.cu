// pkv_tables.cu -- the tables of a step built on the GPU from the requests'
// lengths (pkv_build_tables): new pages from a free list into the page table,
// prefix sums, positions and slots of the new tokens.
//
// With q_b new tokens in a context of n_b, entry b takes
//   need_b = ceil(n_b / ps) - ceil((n_b - q_b) / ps)
// pages, and new token i belongs to the entry b with Q_b <= i < Q_b + q_b,
// Q the exclusive prefix sum of q; its page is free_pages[*free_start + N_b +
// (page index - first new page)], N the exclusive prefix sum of need, or one
// that the entry already had.
//
// A step has few entries and many tokens, so each CTA owns a run of new
// tokens and forms the prefix sums of the whole batch by itself (the lengths
// come from L2), a tile of entries at a time, then finds each token's entry
// by bisection in the tile's sums in shared memory.  Nothing passes between
// CTAs, so one launch does everything; the first CTA alone writes the prefix
// sums and reports errors of the entries.  Bound by latency (the launch, the
// lengths, the scan, the table): 4.5 us for 64 entries with a token each, 7.8 us
// for 256 entries with 278K tokens (3.5 MB written).
#include "pkv_common.cuh"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kPer = 4;                    // entries per thread and tile
constexpr int kTile = kThreads * kPer;

struct Entry {
    int row, len, q, need;
    bool ok;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

__device__ __forceinline__ Entry load_entry(const TablesParams &p, int b, bool report) {
    Entry e;
    e.row = __ldg(p.req_pool_indices + b);
    e.len = __ldg(p.seq_lens + b);
    e.q = p.q_lens ? __ldg(p.q_lens + b) : (e.len > 0);
    int bad = 0;
    e.ok = true;
    if (static_cast<unsigned>(e.row) >= static_cast<unsigned>(p.num_reqs)) e.ok = false, bad = e.row;
    else if (static_cast<unsigned>(e.len) > static_cast<unsigned>(p.max_len)) e.ok = false, bad = e.len;
    else if (static_cast<unsigned>(e.q) > static_cast<unsigned>(e.len)) e.ok = false, bad = e.q;
    if (!e.ok) {
        if (report) record_error(p.err, bad);
        e.len = e.q = 0;
    }
    e.need = e.q ? ceil_div(e.len, p.page_size) - ceil_div(e.len - e.q, p.page_size) : 0;
    return e;
}

__device__ __forceinline__ int clamp31(long long x) { return static_cast<int>(x < 0x7fffffffLL ? x : 0x7fffffffLL); }

// The tokens beyond max_new get no slot, but their pages are taken: they go to
// the table too, which otherwise would keep another request's pages.  Entries b0
// .. b0 + n, by one CTA (out of line: an error's path, off the others' code).
__device__ __noinline__ void enter_pages_without_slots(const TablesParams &p, const int *tok_off, const int *page_off, int b0, int n) {
    const int lane = threadIdx.x & 31;
    for (int a = threadIdx.x >> 5; a < n; a += kThreads / 32) {
        const Entry x = load_entry(p, b0 + a, false);
        const int old = x.len - x.q, fresh = ceil_div(old, p.page_size);
        const long long kept = static_cast<long long>(p.max_new) - tok_off[a] + old;   // positions before it have slots
        const long long from = kept > 0 ? max(static_cast<long long>(fresh), (kept + p.page_size - 1) / p.page_size) : fresh;
        for (long long idx = from + lane; idx < fresh + x.need; idx += 32) {
            const long long at = page_off[a] + (idx - fresh);
            int page = at < p.n_free ? __ldg(p.free_pages + at) : -1;
            if (static_cast<unsigned>(page) >= static_cast<unsigned long long>(p.n_pages)) {
                record_error(p.err, at < p.n_free ? page : -300000LL - (b0 + a));
                page = -1;
            }
            p.req_to_page[static_cast<int64_t>(x.row) * p.max_pages + idx] = page;
        }
    }
}

__global__ void __launch_bounds__(kThreads) build_tables_kernel(const __grid_constant__ TablesParams p) {
    __shared__ int tok_off[kTile];           // first new token of each entry of the tile
    __shared__ int page_off[kTile];          // its first place in the free list
    __shared__ long long warp_sum[kThreads / 32][3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool first = blockIdx.x == 0;
    const int lo = static_cast<int>(min(static_cast<long long>(blockIdx.x) * p.chunk, static_cast<long long>(p.max_new)));
    const int hi = static_cast<int>(min(static_cast<long long>(lo) + p.chunk, static_cast<long long>(p.max_new)));
    int start = __ldg(p.free_start);
    if (static_cast<unsigned>(start) > static_cast<unsigned>(p.n_free)) {
        if (first && tid == 0) record_error(p.err, start);
        start = p.n_free;
    }
    long long toks = 0, pages = start, kvs = 0;   // sums before the tile

    for (int b0 = 0; b0 < p.batch; b0 += kTile) {
        // sums of this thread's entries, then of the threads before it
        Entry e[kPer];
        long long s[3] = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = b0 + tid * kPer + i;
            e[i] = b < p.batch ? load_entry(p, b, first) : Entry{0, 0, 0, 0, true};
            s[0] += e[i].q;
            s[1] += e[i].need;
            s[2] += e[i].len;
        }
        long long inc[3] = {s[0], s[1], s[2]};
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const long long y = __shfl_up_sync(0xffffffffu, inc[k], off);
                if (lane >= off) inc[k] += y;
            }
        }
        __syncthreads();                     // the previous tile's readers are done
        if (lane == 31)
            for (int k = 0; k < 3; ++k) warp_sum[warp][k] = inc[k];
        __syncthreads();
        long long before[3] = {toks, pages, kvs}, total[3] = {toks, pages, kvs};
        for (int w = 0; w < kThreads / 32; ++w)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (w < warp) before[k] += warp_sum[w][k];
                total[k] += warp_sum[w][k];
            }
        long long q_at = before[0] + inc[0] - s[0], n_at = before[1] + inc[1] - s[1], k_at = before[2] + inc[2] - s[2];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = b0 + tid * kPer + i;
            tok_off[tid * kPer + i] = clamp31(q_at);
            page_off[tid * kPer + i] = clamp31(n_at);
            q_at += e[i].q;
            n_at += e[i].need;
            k_at += e[i].len;
            if (first && b < p.batch) {
                if (b == 0) {
                    if (p.kv_indptr) p.kv_indptr[0] = 0;
                    if (p.qo_indptr) p.qo_indptr[0] = 0;
                }
                if (p.kv_indptr) p.kv_indptr[b + 1] = clamp31(k_at);
                if (p.qo_indptr) p.qo_indptr[b + 1] = clamp31(q_at);
            }
        }
        __syncthreads();
        const int t0 = max(lo, clamp31(toks)), t1 = min(hi, clamp31(total[0]));
        const int n_tile = min(kTile, p.batch - b0);
        for (int t = t0 + tid; t < t1; t += kThreads) {
            // the last entry that starts at t or before: the one that holds it
            int a = 0, z = n_tile;
            while (z - a > 1) {
                const int m = (a + z) >> 1;
                if (tok_off[m] <= t) a = m;
                else z = m;
            }
            const Entry x = load_entry(p, b0 + a, false);
            const int old = x.len - x.q;
            const int pos = old + (t - tok_off[a]);
            const int idx = pos / p.page_size, off = pos - idx * p.page_size;
            const int fresh = ceil_div(old, p.page_size);
            int32_t *entry_page = p.req_to_page + static_cast<int64_t>(x.row) * p.max_pages + idx;
            int page = -1;
            const long long at = static_cast<long long>(page_off[a]) + (idx - fresh);
            if (idx >= fresh && at >= p.n_free) {
                record_error(p.err, -300000LL - (b0 + a));
            } else {
                page = idx >= fresh ? __ldg(p.free_pages + at) : *entry_page;
                if (static_cast<unsigned>(page) >= static_cast<unsigned long long>(p.n_pages)) {
                    record_error(p.err, page);
                    page = -1;
                }
            }
            if (off == 0) *entry_page = page;
            const int slot = page < 0 ? -1 : page * p.page_size + off;
            p.out_cache_loc[t] = slot;
            if (p.positions) p.positions[t] = pos;
            if (p.req_to_token) p.req_to_token[static_cast<int64_t>(x.row) * p.max_ctx_len + pos] = slot;
        }
        if (first && total[0] > p.max_new) enter_pages_without_slots(p, tok_off, page_off, b0, n_tile);
        toks = total[0];
        pages = total[1];
        kvs = total[2];
        if (!first && toks >= hi) return;
    }
    if (first && tid == 0) {
        if (p.batch == 0) {
            if (p.kv_indptr) p.kv_indptr[0] = 0;
            if (p.qo_indptr) p.qo_indptr[0] = 0;
        }
        if (toks > p.max_new) record_error(p.err, toks);
        if (kvs > 0x7fffffffLL) record_error(p.err, kvs);
        *p.free_end = static_cast<int>(min(pages, static_cast<long long>(p.n_free)));
    }
}

}  // namespace

cudaError_t launch_build_tables(const TablesParams &p, cudaStream_t s) {
    const unsigned grid = p.max_new > 0 ? static_cast<unsigned>((static_cast<long long>(p.max_new) + p.chunk - 1) / p.chunk) : 1u;
    build_tables_kernel<<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
