// pkv_bounds.cu -- the pages' key bounds of the sparse decode (pkv_page_bounds):
// per page, kv head and channel the minimum and maximum of the keys written,
// brought up to date with a batch of new keys, and the same together with the
// cache write (a sparse decode step).  Bound by the latency of dependent loads
// (slots, then a page's rows eight at a time): 2.4 us for 32 keys; 17.4K keys of 8
// kv heads (40 MB) 12.4 us in a call with other inputs before it, 3.2 TB/s, half
// of the copy rate (14.5 with every slot's neighbours loaded one after the
// other), 7.2 with the rows in L2.  A third of its CTAs hold no token that begins
// a page.
#include "pkv_launch.h"
#include "pkv_sparse.cuh"

namespace pkv {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kBoundsThreads = 128;
constexpr int kRowsAhead = 8;

// A run is a maximal sequence of new tokens in one page, with or without gaps
// between their slots (slots outside the pool, which are errors, are passed
// over).  A CTA takes the runs that start among its block_tokens tokens (and
// follows a run beyond them), so no page is updated by two CTAs; thread c reduces
// 16-byte chunk c of the run's rows.  The bytes of the new keys are read once,
// kRowsAhead rows of consecutive slots in flight per thread.
//
// kWrite: the cache write too (a sparse decode step).  A CTA then first copies
// its own tokens' K and V rows to the pool; the bounds come from the new rows,
// not from the pool, so nothing waits for another CTA's copy, and a step has
// one launch less (2.6 + 3.3 us of kernels apart for one token).
template <typename T, bool kWrite>
__global__ void __launch_bounds__(kBoundsThreads, 8) page_bounds_kernel(const BoundsParams p) {
    griddep_launch();
    const int chunk = blockIdx.y * kBoundsThreads + threadIdx.x;
    const int i_end = min(p.n_new, (static_cast<int>(blockIdx.x) + 1) * p.block_tokens);
    const auto valid = [&](int slot) { return static_cast<unsigned>(slot) < static_cast<unsigned long long>(p.size); };
    // lane l of a warp holds the slot of token base + l: one load for a page or two
    const int lane = threadIdx.x & 31;
    int base = 0, window = 0;
    const auto look = [&](int from) {
        base = from;
        window = __ldg(p.out_cache_loc + max(0, min(from + lane, p.n_new - 1)));
    };
    const auto slot_of = [&](int i) {
        if (i < base || i >= base + 32) look(i);
        return __shfl_sync(0xffffffffu, window, i - base);
    };
    look(blockIdx.x * p.block_tokens - 1);
    if constexpr (kWrite) {
        constexpr int kAhead = 4;
        if (chunk < p.row_chunks) {
            for (int i = blockIdx.x * p.block_tokens; i < i_end; i += kAhead) {
                int slot[kAhead];
                uint4 k[kAhead], v[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t at = static_cast<int64_t>(min(i + u, i_end - 1)) * p.row_chunks + chunk;
                    slot[u] = __ldg(p.out_cache_loc + min(i + u, i_end - 1));
                    k[u] = __ldg(static_cast<const uint4 *>(p.keys) + at);
                    v[u] = __ldg(static_cast<const uint4 *>(p.values) + at);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (i + u >= i_end || !valid(slot[u])) continue;   // the loop below reports a bad slot
                    const int64_t to = (p.layer_row0 + slot[u]) * p.row_chunks + chunk;
                    static_cast<uint4 *>(p.k_buffer)[to] = k[u];
                    static_cast<uint4 *>(p.v_buffer)[to] = v[u];
                }
            }
        }
    }
    constexpr int kNotLooked = -2;
    int before = kNotLooked;                 // the slot of the last token before i that is in the pool, -1: none
    for (int i = blockIdx.x * p.block_tokens; i < i_end;) {
        int loc = slot_of(i);
        if (!valid(loc)) {
            if (chunk == 0) record_error(p.err, loc);
            ++i;
            continue;
        }
        const int page = loc / p.page_size, page0 = page * p.page_size;
        const auto in_page = [&](int slot) { return static_cast<unsigned>(slot - page0) < static_cast<unsigned>(p.page_size); };
        if (before == kNotLooked) {
            before = -1;
            for (int j = i - 1; j >= 0 && before < 0; --j) {
                const int slot = slot_of(j);
                if (valid(slot)) before = slot;
            }
        }
        const bool begins = before < 0 || !in_page(before);
        uint4 *dst = static_cast<uint4 *>(p.page_bounds) + (p.layer_page0 + page) * p.row_chunks * 2 +
                     (chunk / p.head_chunks) * p.head_chunks * 2 + chunk % p.head_chunks;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        bool have = false;                   // lo / hi hold something
        const bool mine = begins && chunk < p.row_chunks;
        if (mine && loc != page0) {
            lo = dst[0];
            hi = dst[p.head_chunks];
            have = true;
        }
        for (;;) {
            // tokens i .. i + n - 1 are in consecutive slots of the page
            const int most = min(p.n_new - i, p.page_size - (loc - page0));
            int n = 1;
            while (n < most) {
                if (i + n < base || i + n >= base + 32) look(i + n);
                const int k = base + lane - i;                    // this lane's token, counted from i
                const unsigned breaks = __ballot_sync(0xffffffffu, k >= n && (k >= most || window != loc + k));
                if (breaks) {
                    n = base + __ffs(breaks) - 1 - i;
                    break;
                }
                n = base + 32 - i;
            }
            n = min(n, most);
            if (mine) {
                const uint4 *row = (kWrite ? static_cast<const uint4 *>(p.keys) + static_cast<int64_t>(i) * p.row_chunks
                                           : static_cast<const uint4 *>(p.k_buffer) + (p.layer_row0 + loc) * p.row_chunks) + chunk;
                if (!have) lo = hi = row[0];
                have = true;
                for (int k = 0; k < n; k += kRowsAhead) {
                    uint4 x[kRowsAhead];
#pragma unroll
                    for (int u = 0; u < kRowsAhead; ++u)
                        if (k + u < n) x[u] = row[static_cast<int64_t>(k + u) * p.row_chunks];
#pragma unroll
                    for (int u = 0; u < kRowsAhead; ++u)
                        if (k + u < n) widen_bounds<T>(lo, hi, x[u], x[u]);
                }
            }
            i += n;
            loc += n;
            before = loc - 1;
            if (!begins) break;              // the CTA before goes on with this page
            int j = i, after = 0;
            while (j < p.n_new && !valid(after = slot_of(j))) ++j;
            if (j >= p.n_new || !in_page(after)) break;
            if (chunk == 0)
                for (int x = i; x < j; ++x) record_error(p.err, __ldg(p.out_cache_loc + x));
            i = j;
            loc = after;
        }
        if (mine) {
            dst[0] = lo;
            dst[p.head_chunks] = hi;
        }
    }
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsParams &p, cudaStream_t s) {
    if (p.n_new == 0) return cudaSuccess;
    const dim3 grid((p.n_new + p.block_tokens - 1) / p.block_tokens, (p.row_chunks + kBoundsThreads - 1) / kBoundsThreads);
    if (p.values) {
        if (p.dtype == PKV_BF16) page_bounds_kernel<bf16, true><<<grid, kBoundsThreads, 0, s>>>(p);
        else page_bounds_kernel<float, true><<<grid, kBoundsThreads, 0, s>>>(p);
    } else {
        if (p.dtype == PKV_BF16) page_bounds_kernel<bf16, false><<<grid, kBoundsThreads, 0, s>>>(p);
        else page_bounds_kernel<float, false><<<grid, kBoundsThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace pkv
