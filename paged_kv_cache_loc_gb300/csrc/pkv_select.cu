// pkv_select.cu -- which pages a sparse decode attends to: the pages' key
// bounds (pkv_page_bounds) and the selection by them (pkv_select_pages).
//
// Bounds: per page, kv head and channel the minimum and maximum of the keys
// written.  The score of a page for a query q is the largest product that q
// can have with any key inside the bounds,
//   sum_c max(q_c lo_c, q_c hi_c) = q- . lo + q+ . hi   (q- <= 0 <= q+, q = q- + q+),
// maximised over the G query heads of the group.
//
// The selection must not depend on how a sum was rounded, so it is decided in
// two steps.  The score pass computes 32-bit scores s with |s - s*| <= e,
// where s* is the exact score and, for the n = 2 D (or D) terms of a sum,
//   e = kScoreEps * max_h sum_c |q[h, c]| * max |bound|  >=  n 2^-23 sum |terms|,
// kScoreEps = 2^-14 covering n = 256 terms with every partial sum truncated
// to 24 bits (2^-15) twice over.  With T the 32-bit score of rank
// k, a page with s > T + 2e is in and one with s < T - 2e is out whatever the
// rounding was; the few in between are scored again in 64 bits and ranked by
// (score, page).
#include "pkv_common.cuh"
#include "pkv_launch.h"

namespace pkv {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// ---------------------------------------------------------------------------
// Key bounds
// ---------------------------------------------------------------------------

// Minimum / maximum that keep a NaN.
__device__ __forceinline__ uint32_t min_word(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_word(uint32_t a, uint32_t b, float) {
    return __float_as_uint(min_nan(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b, float) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
}
template <typename T>
__device__ __forceinline__ void widen_bounds(uint4 &lo, uint4 &hi, const uint4 &l, const uint4 &h) {
    lo = make_uint4(min_word(lo.x, l.x, T{}), min_word(lo.y, l.y, T{}), min_word(lo.z, l.z, T{}), min_word(lo.w, l.w, T{}));
    hi = make_uint4(max_word(hi.x, h.x, T{}), max_word(hi.y, h.y, T{}), max_word(hi.z, h.z, T{}), max_word(hi.w, h.w, T{}));
}

constexpr int kBoundsThreads = 128;
constexpr int kRowsAhead = 8;

// A run is a maximal sequence of new tokens in consecutive slots of one page
// (slots outside the pool, which are errors, are passed over).  A CTA takes the
// runs that start among its block_tokens tokens (and follows a run beyond
// them); thread c reduces 16-byte chunk c of the run's rows.  The bytes of the
// new keys are read once, kRowsAhead rows in flight per thread.
//
// kWrite: the cache write too (a sparse decode step).  A CTA then first copies
// its own tokens' K and V rows to the pool; the bounds come from the new rows,
// not from the pool, so nothing waits for another CTA's copy, and a step has
// one launch less (2.6 + 3.3 us of kernels apart for one token).
template <typename T, bool kWrite>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const BoundsParams p) {
    griddep_launch();
    const int chunk = blockIdx.y * kBoundsThreads + threadIdx.x;
    const int i_end = min(p.n_new, (static_cast<int>(blockIdx.x) + 1) * p.block_tokens);
    const auto valid = [&](int slot) { return static_cast<unsigned>(slot) < static_cast<unsigned long long>(p.size); };
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
    for (int i = blockIdx.x * p.block_tokens; i < i_end;) {
        int loc = __ldg(p.out_cache_loc + i);
        if (!valid(loc)) {
            if (chunk == 0) record_error(p.err, loc);
            ++i;
            continue;
        }
        const int page = loc / p.page_size;
        int off = loc - page * p.page_size;
        bool begins = off == 0;
        if (!begins) {
            int j = i - 1;
            while (j >= 0 && !valid(__ldg(p.out_cache_loc + j))) --j;
            begins = j < 0 || __ldg(p.out_cache_loc + j) != loc - 1;
        }
        uint4 *dst = static_cast<uint4 *>(p.page_bounds) + (p.layer_page0 + page) * p.row_chunks * 2 +
                     (chunk / p.head_chunks) * p.head_chunks * 2 + chunk % p.head_chunks;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        bool have = false;                   // lo / hi hold something
        const bool mine = begins && chunk < p.row_chunks;
        if (mine && off != 0) {
            lo = dst[0];
            hi = dst[p.head_chunks];
            have = true;
        }
        for (;;) {
            // tokens i .. i + n - 1 are in consecutive slots of the page
            const int most = min(p.n_new - i, p.page_size - off);
            int n = 1;
            for (;;) {
                const int at = n + static_cast<int>(threadIdx.x & 31);
                const bool next = at < most && __ldg(p.out_cache_loc + i + at) == loc + at;
                const unsigned breaks = __ballot_sync(0xffffffffu, !next);
                n += breaks ? __ffs(breaks) - 1 : 32;
                if (breaks) break;
            }
            if (mine) {
                const uint4 *row = (kWrite ? static_cast<const uint4 *>(p.keys) + static_cast<int64_t>(i) * p.row_chunks
                                           : static_cast<const uint4 *>(p.k_buffer) + (p.layer_row0 + loc) * p.row_chunks) + chunk;
                if (!have) lo = hi = row[0];
                have = true;
                for (int k = 0; k < n; k += kRowsAhead) {
                    uint4 x[kRowsAhead];
#pragma unroll
                    for (int u = 0; u < kRowsAhead; ++u) x[u] = row[static_cast<int64_t>(min(k + u, n - 1)) * p.row_chunks];
#pragma unroll
                    for (int u = 0; u < kRowsAhead; ++u) widen_bounds<T>(lo, hi, x[u], x[u]);
                }
            }
            i += n;
            off += n;
            loc += n;
            if (!begins || off == p.page_size) break;
            int j = i;
            while (j < p.n_new && !valid(__ldg(p.out_cache_loc + j))) ++j;
            if (j == i || j >= p.n_new || __ldg(p.out_cache_loc + j) != loc) break;
            if (chunk == 0)
                for (int x = i; x < j; ++x) record_error(p.err, __ldg(p.out_cache_loc + x));
            i = j;
        }
        if (mine) {
            dst[0] = lo;
            dst[p.head_chunks] = hi;
        }
    }
}

// ---------------------------------------------------------------------------
// Scores
// ---------------------------------------------------------------------------

constexpr float kScoreEps = 6.103515625e-5f;   // 2^-14
constexpr float kScoreTiny = 1e-35f;           // 256 products lost below the smallest normal number, doubled

// 4-byte words of a bounds or q row, widened.
__device__ __forceinline__ void widen16(const uint4 &w, float (&x)[8], bf16) {
    x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
}
__device__ __forceinline__ void widen16(const uint4 &w, float (&x)[4], float) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
}

// Number of pages of entry b (0 with a request row out of range); the row.
__device__ __forceinline__ int entry_pages(const SelectParams &p, int b, int *row, bool report) {
    const int r = __ldg(p.req_pool_indices + b);
    int n = __ldg(p.seq_lens + b);
    if (static_cast<unsigned>(r) >= static_cast<unsigned>(p.num_reqs)) {
        if (report) record_error(p.err, r);
        *row = 0;
        return 0;
    }
    *row = r;
    if (n < 0 || n > p.max_len) {
        if (report) record_error(p.err, n);
        n = n < 0 ? 0 : p.max_len;
    }
    return n / p.page_size + (n % p.page_size != 0);
}

__device__ __forceinline__ long long page_at(const SelectParams &p, int row, int i) {
    const int pg = __ldg(p.req_to_page + static_cast<int64_t>(row) * p.max_pages + i);
    if (static_cast<unsigned>(pg) < static_cast<unsigned long long>(p.n_pages)) return pg;
    record_error(p.err, pg);
    return 0;
}

constexpr int kScoreWarps = 4;

// CUDA-core scores: a warp takes kScoreGroup pages, eight lanes to a page,
// each lane the 16-byte chunks c = lane % 8, c + 8, ... of the page's rows.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kScoreWarps * 32) score_pages_kernel(const SelectParams p) {
    constexpr int kElems = 16 / Elem<T>::bytes;
    constexpr int kChunks = D / kElems;              // 16-byte chunks per row
    __shared__ float q[G][D];
    griddep_launch();
    const int g = blockIdx.y, b = blockIdx.z;
    int row;
    const int n = entry_pages(p, b, &row, false);
    for (int i = threadIdx.x; i < G * D; i += kScoreWarps * 32)
        q[i / D][i % D] = Elem<T>::to_f(static_cast<const T *>(p.q)[(static_cast<int64_t>(b) * p.n_heads + g * G) * D + i]);
    __syncthreads();
    if (p.pdl) griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7;
    const int group = blockIdx.x * kScoreWarps + warp;
    if (n <= p.top_k || group * kScoreGroup >= n) return;
    float biggest = 0.f;
    const int64_t unit = static_cast<int64_t>(b) * p.n_kv_heads + g;
#pragma unroll 1
    for (int i = 0; i < kScoreGroup; i += 4) {
        const int pg = group * kScoreGroup + i + (lane >> 3);
        const int pc = min(pg, n - 1);
        const uint4 *lo = static_cast<const uint4 *>(p.page_bounds) +
                          ((p.layer_page0 + page_at(p, row, pc)) * p.n_kv_heads + g) * 2 * kChunks;
        float s[G];
#pragma unroll
        for (int h = 0; h < G; ++h) s[h] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; c += 8) {
            float l[kElems], u[kElems];
            widen16(__ldg(lo + c + sub), l, T{});
            widen16(__ldg(lo + kChunks + c + sub), u, T{});
#pragma unroll
            for (int x = 0; x < kElems; ++x) {
                biggest = max_nan(biggest, max_nan(fabsf(l[x]), fabsf(u[x])));
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float qv = q[h][(c + sub) * kElems + x];
                    s[h] = fmaf(qv, qv >= 0.f ? u[x] : l[x], s[h]);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
            for (int off = 4; off >= 1; off >>= 1) s[h] += __shfl_xor_sync(0xffffffffu, s[h], off);
        float best = s[0];
#pragma unroll
        for (int h = 1; h < G; ++h) best = max_nan(best, s[h]);
        if (sub == 0 && pg < n) p.scores[unit * p.page_cap + pg] = best;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) biggest = max_nan(biggest, __shfl_xor_sync(0xffffffffu, biggest, off));
    if (lane == 0) p.group_max[unit * (p.page_cap / kScoreGroup) + group] = biggest;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Tensor-core scores (bf16): the score is a product, [hi, lo] of 16 pages times
// [q+, q-] of the group's heads, so a warp takes kScoreGroup = 16 pages as the
// rows and the heads as the 8 columns of m16n8k16.  A dot product may take its
// terms in any order, so lane (r, t) = (lane / 4, lane % 4) supplies the
// 16-byte chunks t, t + 4, ... of rows r and r + 8 (and of head r) straight
// from memory: four lanes read 64 contiguous bytes, nothing is staged, and a
// warp has all of its 8 KB (D = 128) in flight at once.
template <int D, int G>
__global__ void __launch_bounds__(kScoreWarps * 32) score_pages_mma_kernel(const SelectParams p) {
    constexpr int kChunks = D / 8, kOwn = kChunks / 4;
    griddep_launch();
    const int g = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
    const int group = blockIdx.x * kScoreWarps + warp;
    int row;
    const int n = entry_pages(p, b, &row, false);
    if (n <= p.top_k || group * kScoreGroup >= n) {
        if (p.pdl) griddep_wait();
        return;
    }
    uint4 q[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        q[j] = r < G ? __ldg(static_cast<const uint4 *>(p.q) + (static_cast<int64_t>(b) * p.n_heads + g * G + r) * kChunks + t + 4 * j)
                     : make_uint4(0, 0, 0, 0);
    int page = static_cast<int>(page_at(p, row, min(group * kScoreGroup + (lane & 15), n - 1)));
    if (p.pdl) griddep_wait();
    const uint4 *base = static_cast<const uint4 *>(p.page_bounds) + t;
    const uint4 *r0 = base + ((p.layer_page0 + __shfl_sync(0xffffffffu, page, r)) * p.n_kv_heads + g) * 2 * kChunks;
    const uint4 *r1 = base + ((p.layer_page0 + __shfl_sync(0xffffffffu, page, r + 8)) * p.n_kv_heads + g) * 2 * kChunks;
    uint4 l0[kOwn], l1[kOwn], h0[kOwn], h1[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        l0[j] = __ldg(r0 + 4 * j);
        l1[j] = __ldg(r1 + 4 * j);
        h0[j] = __ldg(r0 + kChunks + 4 * j);
        h1[j] = __ldg(r1 + kChunks + 4 * j);
    }
    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
    uint4 most = h0[0], least = l0[0];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const uint4 qn = make_uint4(min_word(q[j].x, 0, bf16{}), min_word(q[j].y, 0, bf16{}), min_word(q[j].z, 0, bf16{}), min_word(q[j].w, 0, bf16{}));
        const uint4 qp = make_uint4(max_word(q[j].x, 0, bf16{}), max_word(q[j].y, 0, bf16{}), max_word(q[j].z, 0, bf16{}), max_word(q[j].w, 0, bf16{}));
        mma16816(x, l0[j].x, l1[j].x, l0[j].y, l1[j].y, qn.x, qn.y);
        mma16816(y, h0[j].x, h1[j].x, h0[j].y, h1[j].y, qp.x, qp.y);
        mma16816(x, l0[j].z, l1[j].z, l0[j].w, l1[j].w, qn.z, qn.w);
        mma16816(y, h0[j].z, h1[j].z, h0[j].w, h1[j].w, qp.z, qp.w);
        widen_bounds<bf16>(least, most, l0[j], h0[j]);
        widen_bounds<bf16>(least, most, l1[j], h1[j]);
    }
    // rows r and r + 8, heads 2t and 2t + 1
    float s0 = -INFINITY, s1 = -INFINITY;
    if (2 * t < G) {
        s0 = x[0] + y[0];
        s1 = x[2] + y[2];
    }
    if (2 * t + 1 < G) {
        s0 = max_nan(s0, x[1] + y[1]);
        s1 = max_nan(s1, x[3] + y[3]);
    }
    const uint32_t hi = max_word(max_word(most.x, most.y, bf16{}), max_word(most.z, most.w, bf16{}), bf16{});
    const uint32_t lo = min_word(min_word(least.x, least.y, bf16{}), min_word(least.z, least.w, bf16{}), bf16{});
    float biggest = max_nan(max_nan(bf16lo(hi), bf16hi(hi)), -min_nan(bf16lo(lo), bf16hi(lo)));
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
        s0 = max_nan(s0, __shfl_xor_sync(0xffffffffu, s0, off));
        s1 = max_nan(s1, __shfl_xor_sync(0xffffffffu, s1, off));
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) biggest = max_nan(biggest, __shfl_xor_sync(0xffffffffu, biggest, off));
    const int64_t unit = static_cast<int64_t>(b) * p.n_kv_heads + g;
    float *out = p.scores + unit * p.page_cap + group * kScoreGroup;      // page_cap is whole groups
    if (t == 0) {
        out[r] = s0;
        out[r + 8] = s1;
    }
    if (lane == 0) p.group_max[unit * (p.page_cap / kScoreGroup) + group] = biggest;
}

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kUndecided = 512;          // scored in 64 bits from a list; more: by radix passes

// Order-preserving integer keys; NaN above every number, -0 = +0.
__device__ __forceinline__ uint32_t key32(float s) {
    if (s != s) return 0xffffffffu;
    const uint32_t u = __float_as_uint(s + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unkey32(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long key64(double s) {
    if (s != s) return ~0ull;
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s + 0.0));
    return u >> 63 ? ~u : u | (1ull << 63);
}

template <int D, int G>
struct SelShared {
    float q[G][D];
    int hist[kBins];
    unsigned long long warp_sum[kSelWarps];
    uint32_t lo[kSelWarps], hi[kSelWarps], big[kSelWarps];
    int bin, above;
    int und_page[kUndecided], und_phys[kUndecided];
    long long und_key[kUndecided];
    uint32_t und_in[kUndecided / 32];
};

// Inclusive scan over the block of a whole number per thread.
template <typename N>
__device__ __forceinline__ N block_scan(unsigned long long *warp_sum, N v, N *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    N w = lane < kSelWarps ? static_cast<N>(warp_sum[lane]) : N(0);
#pragma unroll
    for (int off = 1; off < kSelWarps; off <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, kSelWarps - 1);
    const N before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return warp > 0 ? v + before : v;
}

// The bin (from the top) that holds rank `rank` (1-based) of the histogram of
// kBins bins: sh.bin, and sh.above = the count in higher bins.
template <int D, int G>
__device__ __forceinline__ void find_bin(SelShared<D, G> &sh, int rank) {
    constexpr int kPer = kBins / kSelThreads;
    const int top = kBins - 1 - static_cast<int>(threadIdx.x) * kPer;   // this thread: top, top - 1, ...
    int c[kPer], own = 0, total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) own += c[k] = sh.hist[top - k];
    const int inc = block_scan(sh.warp_sum, own, &total);
    int before = inc - own;
    if (before < rank && rank <= inc) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (before < rank && rank <= before + c[k]) {
                sh.bin = top - k;
                sh.above = before;
            }
            before += c[k];
        }
    }
    __syncthreads();
}

// The 64-bit key of a page's score for query head h, by a warp: lane partial
// sums in a fixed order, so equal bounds give equal keys.
template <typename T, int D>
__device__ __forceinline__ unsigned long long exact_head_key(const SelectParams &p, const float *q, int64_t bounds_row) {
    const int lane = threadIdx.x & 31;
    const T *lo = static_cast<const T *>(p.page_bounds) + bounds_row * 2 * D;
    float l[D / 32], u[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        l[c] = Elem<T>::to_f(lo[c * 32 + lane]);
        u[c] = Elem<T>::to_f(lo[D + c * 32 + lane]);
    }
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const float qv = q[c * 32 + lane];
        s = fma(static_cast<double>(qv), static_cast<double>(qv >= 0.f ? u[c] : l[c]), s);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return key64(s);
}

template <typename T, int D, int G>
__device__ __forceinline__ unsigned long long exact_key(const SelectParams &p, const SelShared<D, G> &sh, int row, int g, int pg) {
    const int64_t at = (p.layer_page0 + page_at(p, row, pg)) * p.n_kv_heads + g;
    unsigned long long best = 0;
#pragma unroll 1
    for (int h = 0; h < G; ++h) best = max(best, exact_head_key<T, D>(p, sh.q[h], at));
    return best;
}

// Largest sum_c |q[h, c]| over the heads, every warp by itself.
template <int D, int G>
__device__ __forceinline__ float query_norm(const SelShared<D, G> &sh) {
    const int lane = threadIdx.x & 31;
    float norm = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < D; c += 32) s += fabsf(sh.q[h][c + lane]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        norm = max_nan(norm, s);
    }
    return norm;
}

// Scores in 64-bit fixed point.  With |score| <= norm * big < 2^e, a term
// counts in units of 2^(e - 61): a bf16 product is exact in fp32, an fp32 one
// is taken as its rounding and the remainder, and integer sums do not round,
// so the order of the terms does not matter.  Each term is off by half a unit
// at most, 2^-62 of the bound, where a sum in fp64 rounds to 2^-53 of the
// partial sums; fp64 arithmetic itself is too slow on this chip (17 us of a
// selection went there).  For scale exponents inside fp32's range; the general
// path takes fp64 otherwise.
__device__ __forceinline__ bool fixed_point_scale(float norm, float big, float *scale) {
    int a = 0, b = 0;
    frexpf(norm, &a);
    frexpf(big, &b);
    const int e = a + b + 1;                 // one more: norm is a rounded sum
    *scale = ldexpf(1.f, 61 - (e < -40 ? -40 : e > 120 ? 120 : e));
    return e >= -40 && e <= 120;
}

// A page's fixed-point score for one query head, by eight lanes of a warp (sub =
// lane % 8), each the 16-byte chunks sub, sub + 8, ...
template <typename T, int D>
__device__ __forceinline__ long long fixed_score(const SelectParams &p, const float *q, int64_t bounds_row, float scale, int sub) {
    constexpr int kElems = 16 / Elem<T>::bytes, kChunks = D / kElems;
    const uint4 *lo = static_cast<const uint4 *>(p.page_bounds) + bounds_row * 2 * kChunks + sub;
    uint4 l[kChunks / 8], u[kChunks / 8];
#pragma unroll
    for (int c = 0; c < kChunks / 8; ++c) {
        l[c] = __ldg(lo + 8 * c);
        u[c] = __ldg(lo + kChunks + 8 * c);
    }
    long long s = 0;
#pragma unroll
    for (int c = 0; c < kChunks / 8; ++c) {
        float a[kElems], b[kElems];
        widen16(l[c], a, T{});
        widen16(u[c], b, T{});
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
            const float qv = q[(8 * c + sub) * kElems + e], x = qv >= 0.f ? b[e] : a[e], prod = qv * x;
            s += __float2ll_rn(prod * scale);
            if constexpr (Elem<T>::bytes == 4) s += __float2ll_rn(fmaf(qv, x, -prod) * scale);
        }
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

constexpr long long kLeastKey = -0x7fffffffffffffffLL - 1;

// Ranks the `n` <= kUndecided pages of sh.und_page by their fixed-point scores
// and sets the bits of sh.und_in for the first `need` of them.  On entry
// sh.und_phys holds their physical pages and sh.und_key is kLeastKey.
template <typename T, int D, int G>
__device__ __forceinline__ void rank_undecided(const SelectParams &p, SelShared<D, G> &sh, int g, int n, int need, float scale) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int x0 = warp * 4; x0 < n * G; x0 += kSelWarps * 4) {    // eight lanes per (page, head)
        const int x = min(x0 + lane / 8, n * G - 1), k = x / G, h = x % G;
        const int64_t at = (p.layer_page0 + sh.und_phys[k]) * p.n_kv_heads + g;
        const long long key = fixed_score<T, D>(p, sh.q[h], at, scale, lane % 8);
        if (lane % 8 == 0) atomicMax(&sh.und_key[k], key);
    }
    __syncthreads();
    static_assert(kUndecided <= kSelThreads, "one undecided page per thread");
    bool in = false;
    if (tid < n) {
        const long long key = sh.und_key[tid];
        const int pg = sh.und_page[tid];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.und_key[j] > key || (sh.und_key[j] == key && sh.und_page[j] < pg);
        in = rank < need;
    }
    const unsigned bits = __ballot_sync(0xffffffffu, in);
    if (lane == 0 && warp < kUndecided / 32) sh.und_in[warp] = bits;
    __syncthreads();
}

// The threshold's bin, the error bound on both sides included, as keys [lo, hi]
// of the 32-bit scores, narrowed until at most kUndecided pages lie in it or a
// bin is one key.  sh.hist is zero on entry.  each(f) calls f(key) for this
// thread's candidates.
struct Threshold {
    uint32_t lo, hi;
    int in, mid;                             // candidates above it and inside
    int in_before, mid_before;               // of the threads before this one
};
template <int D, int G, typename Each>
__device__ __forceinline__ Threshold find_threshold(SelShared<D, G> &sh, uint32_t lo, uint32_t hi, int rank, float slack, Each each) {
    const int tid = threadIdx.x;
    for (;;) {
        const int shift = max(0, 32 - __clz(hi - lo) - 11);
        each([&](uint32_t k) {
            if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1);
        });
        __syncthreads();
        find_bin(sh, rank);
        rank -= sh.above;
        lo += static_cast<uint32_t>(sh.bin) << shift;
        hi = min(hi, lo + ((1u << shift) - 1u));
        Threshold x;
        x.lo = key32(unkey32(lo) - slack);
        x.hi = key32(unkey32(hi) + slack);
        unsigned long long both = 0;
        each([&](uint32_t k) { both += k > x.hi ? 1ull << 32 : k >= x.lo ? 1ull : 0ull; });
        unsigned long long total;
        const unsigned long long before = block_scan(sh.warp_sum, both, &total) - both;
        x.in = static_cast<int>(total >> 32);
        x.mid = static_cast<int>(total);
        x.in_before = static_cast<int>(before >> 32);
        x.mid_before = static_cast<int>(before);
        if (x.mid <= kUndecided || shift == 0) return x;
        for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
        __syncthreads();
    }
}

// The general path: scores stay in memory and are read in every pass; decided
// pages are marked there by NaN (in: its key is above all) and -inf.  For contexts of more pages than the
// registers hold, and where more than kUndecided pages are undecided.
template <typename T, int D, int G>
__device__ __noinline__ void select_general(const SelectParams &p, SelShared<D, G> &sh, int row, int g, int n, float *score, int32_t *sel,
                                            uint32_t klo, uint32_t khi, float slack, bool finite, float scale) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float kIn = __uint_as_float(0x7fffffffu);
    const int c0 = p.n_first, m = n - p.n_first - p.n_last, keep = p.top_k - p.n_first - p.n_last;
    score += c0;
    Threshold th{0u, 0xffffffffu, 0, m, 0, 0};
    const auto each = [&](auto f) {
        for (int i = tid; i < m; i += kSelThreads) f(key32(score[i]));
    };
    if (finite) th = find_threshold(sh, klo, khi, keep, slack, each);
    const auto inside = [&](float s) { return key32(s) >= th.lo && key32(s) <= th.hi; };
    const int need = keep - th.in, undecided = th.mid;
    if (need < undecided) {
        if (finite && undecided <= kUndecided) {
            if (tid == 0) sh.bin = 0;
            __syncthreads();
            for (int i = tid; i < m; i += kSelThreads)
                if (inside(score[i])) {
                    const int k = atomicAdd(&sh.bin, 1);
                    sh.und_page[k] = c0 + i;
                    sh.und_phys[k] = static_cast<int>(page_at(p, row, c0 + i));
                    sh.und_key[k] = kLeastKey;
                }
            __syncthreads();
            rank_undecided<T, D, G>(p, sh, g, undecided, need, scale);
            for (int k = tid; k < undecided; k += kSelThreads)
                score[sh.und_page[k] - c0] = sh.und_in[k / 32] >> (k % 32) & 1 ? kIn : -INFINITY;
        } else {
            // Many pages within rounding of the threshold (pages that are
            // alike, or scores that are not finite): radix selection on the
            // 64-bit keys, computed again in each of its eight passes.
            unsigned long long prefix = 0;
            int rank = need;
            for (int byte = 7; byte >= 0; --byte) {
                for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
                __syncthreads();
                for (int i = warp; i < m; i += kSelWarps) {
                    if (!inside(score[i])) continue;
                    const unsigned long long x = exact_key<T, D, G>(p, sh, row, g, c0 + i);
                    if (lane == 0 && (byte == 7 || (x >> (8 * byte + 8)) == (prefix >> (8 * byte + 8))))
                        atomicAdd(&sh.hist[(x >> (8 * byte)) & 255], 1);
                }
                __syncthreads();
                find_bin(sh, rank);
                rank -= sh.above;
                prefix |= static_cast<unsigned long long>(sh.bin) << (8 * byte);
                __syncthreads();
            }
            // keys above the prefix are in, and the first `rank` that equal it
            int equal = 0;
            for (int i0 = 0; i0 < m; i0 += kSelWarps) {
                const int i = i0 + warp;
                const bool mine = i < m && inside(score[i]);
                const unsigned long long x = mine ? exact_key<T, D, G>(p, sh, row, g, c0 + i) : 0;
                int t;
                const int at = equal + block_scan(sh.warp_sum, static_cast<int>(mine && x == prefix && lane == 0), &t);
                if (mine && lane == 0) score[i] = x > prefix || (x == prefix && at <= rank) ? kIn : -INFINITY;
                equal += t;
            }
        }
        __syncthreads();
    }
    // in ascending order: pages above the bin, and of the bin those marked in
    // (all of it where its pages are all needed; with scores that are not
    // finite every page is marked)
    const uint32_t least = need >= undecided ? th.lo : finite ? th.hi + 1 : key32(kIn);
    const int per = (m + kSelThreads - 1) / kSelThreads;
    const int i0 = min(m, tid * per), i1 = min(m, i0 + per);
    int mine = 0, t;
    for (int i = i0; i < i1; ++i) mine += key32(score[i]) >= least;
    int at = p.n_first + block_scan(sh.warp_sum, mine, &t) - mine;
    for (int i = i0; i < i1; ++i)
        if (key32(score[i]) >= least) sel[at++] = c0 + i;
}

// One CTA per (kv head, entry).  Up to kSelThreads * kOwn pages, thread i keeps
// the keys of pages kOwn * i ... in registers: the scores are read once, and
// every later pass (range, histogram, counts, output) is on registers with one
// block-wide scan.  What bounds it is the chain of these passes (latency); the
// bytes are few.
template <typename T, int D, int G, int kOwn>
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(const SelectParams p) {
    __shared__ SelShared<D, G> sh;
    griddep_launch();
    const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t unit = static_cast<int64_t>(b) * p.n_kv_heads + g;
    for (int i = tid; i < G * D; i += kSelThreads)
        sh.q[i / D][i % D] = Elem<T>::to_f(static_cast<const T *>(p.q)[(static_cast<int64_t>(b) * p.n_heads + g * G) * D + i]);
    for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
    int row;
    const int n = entry_pages(p, b, &row, g == 0 && tid == 0);
    int32_t *sel = p.sel + unit * p.top_k;
    if (tid == 0) p.sel_counts[unit] = min(n, p.top_k);
    if (n <= p.top_k) {
        for (int i = tid; i < p.top_k; i += kSelThreads) sel[i] = i < n ? i : -1;
        griddep_wait();
        return;
    }
    const int keep = p.top_k - p.n_first - p.n_last, c1 = n - p.n_last;   // candidates: pages n_first .. c1 - 1
    for (int i = tid; i < p.n_first; i += kSelThreads) sel[i] = i;
    for (int i = tid; i < p.n_last; i += kSelThreads) sel[p.top_k - p.n_last + i] = c1 + i;
    // the physical pages of this thread's pages, in case they are undecided
    const int mine = tid * kOwn;                                  // this thread's first page
    int phys[kOwn > 0 ? kOwn : 1];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        phys[i] = mine + i < n ? __ldg(p.req_to_page + static_cast<int64_t>(row) * p.max_pages + mine + i) : 0;
        if (static_cast<unsigned>(phys[i]) >= static_cast<unsigned long long>(p.n_pages)) phys[i] = 0;   // the score pass reported it
    }
    __syncthreads();
    const float norm = query_norm(sh);
    griddep_wait();                                               // the scores
    if (keep == 0) return;
    float *score = p.scores + unit * p.page_cap;
    const float *gmax = p.group_max + unit * (p.page_cap / kScoreGroup);

    float big = 0.f;
    for (int i = tid; i < (n + kScoreGroup - 1) / kScoreGroup; i += kSelThreads) big = max_nan(big, gmax[i]);
    uint32_t klo = 0xffffffffu, khi = 0;
    uint32_t key[kOwn > 0 ? kOwn : 1];
    const auto owned = [&](int i) { return mine + i >= p.n_first && mine + i < c1; };
    if constexpr (kOwn > 0) {
        if (mine < n) {                                           // page_cap is a multiple of kScoreGroup
#pragma unroll
            for (int i = 0; i < kOwn; i += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(score + mine + i);
                key[i] = key32(x.x);
                key[i + 1] = key32(x.y);
                key[i + 2] = key32(x.z);
                key[i + 3] = key32(x.w);
            }
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (owned(i)) {
                klo = min(klo, key[i]);
                khi = max(khi, key[i]);
            }
    } else {
        for (int i = p.n_first + tid; i < c1; i += kSelThreads) {
            const uint32_t k = key32(score[i]);
            klo = min(klo, k);
            khi = max(khi, k);
        }
    }
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    // |bounds| and NaN order like their bits
    const uint32_t big_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(big) & 0x7fffffffu);
    if (lane == 0) {
        sh.lo[warp] = klo;
        sh.hi[warp] = khi;
        sh.big[warp] = big_bits;
    }
    __syncthreads();
    klo = __reduce_min_sync(0xffffffffu, sh.lo[lane % kSelWarps]);
    khi = __reduce_max_sync(0xffffffffu, sh.hi[lane % kSelWarps]);
    big = __uint_as_float(__reduce_max_sync(0xffffffffu, sh.big[lane % kSelWarps]));
    const float slack = 2.f * kScoreEps * norm * big + kScoreTiny;   // 2e
    float scale = 0.f;
    const bool finite = klo > key32(-INFINITY) && khi < key32(INFINITY) && slack < INFINITY && fixed_point_scale(norm, big, &scale);
    if (kOwn == 0 || !finite) {
        select_general<T, D, G>(p, sh, row, g, n, score, sel, klo, khi, slack, finite, scale);
        return;
    }
    if constexpr (kOwn > 0) {
        const auto each = [&](auto f) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                if (owned(i)) f(key[i]);
        };
        const Threshold th = find_threshold(sh, klo, khi, keep, slack, each);
        const int need = keep - th.in;
        const bool whole = need >= th.mid;                        // the bin's pages are all needed
        if (!whole) {
            if (th.mid > kUndecided) {
                for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
                __syncthreads();
                select_general<T, D, G>(p, sh, row, g, n, score, sel, klo, khi, slack, finite, scale);
                return;
            }
            int k = th.mid_before;
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                if (owned(i) && key[i] >= th.lo && key[i] <= th.hi) {
                    sh.und_page[k] = mine + i;
                    sh.und_phys[k] = phys[i];
                    sh.und_key[k++] = kLeastKey;
                }
            __syncthreads();
            rank_undecided<T, D, G>(p, sh, g, th.mid, need, scale);
        }
        // in ascending order; the list of undecided pages is ascending too
        int at = p.n_first + th.in_before, k = th.mid_before;
        if (whole) {
            at += k;
        } else {
            for (int w = 0; w < k / 32; ++w) at += __popc(sh.und_in[w]);
            at += k % 32 ? __popc(sh.und_in[k / 32] & ((1u << (k % 32)) - 1u)) : 0;
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (!owned(i) || key[i] < th.lo) continue;
            bool in = true;
            if (key[i] <= th.hi) {
                in = whole || (sh.und_in[k / 32] >> (k % 32) & 1);
                ++k;
            }
            if (in) sel[at++] = mine + i;
        }
    }
}

template <typename T, int D, int G>
cudaError_t launch_select(const SelectParams &p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const bool scored = p.scores != nullptr;
    if (scored) {
        const int groups = p.page_cap / kScoreGroup;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((groups + kScoreWarps - 1) / kScoreWarps, p.n_kv_heads, p.batch);
        cfg.blockDim = dim3(kScoreWarps * 32);
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = p.pdl ? 1 : 0;
        cudaError_t e;
        if constexpr (Elem<T>::bytes == 2) e = cudaLaunchKernelEx(&cfg, score_pages_mma_kernel<D, G>, p);
        else e = cudaLaunchKernelEx(&cfg, score_pages_kernel<T, D, G>, p);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.n_kv_heads, p.batch);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = scored || p.pdl ? 1 : 0;
    // pages per thread that the longest context needs; beyond eight the scores
    // stay in memory
    if (p.page_cap <= 4 * kSelThreads) return cudaLaunchKernelEx(&cfg, select_pages_kernel<T, D, G, 4>, p);
    if (p.page_cap <= 8 * kSelThreads) return cudaLaunchKernelEx(&cfg, select_pages_kernel<T, D, G, 8>, p);
    return cudaLaunchKernelEx(&cfg, select_pages_kernel<T, D, G, 0>, p);
}

template <typename T, int D>
cudaError_t launch_select_g(const SelectParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return launch_select<T, D, 1>(p, s);
        case 2: return launch_select<T, D, 2>(p, s);
        case 4: return launch_select<T, D, 4>(p, s);
        case 8: return launch_select<T, D, 8>(p, s);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace

bool sparse_supported(int dtype, int head_dim, int group) {
    return (dtype == PKV_F32 || dtype == PKV_BF16) && (head_dim == 64 || head_dim == 128) &&
           (group == 1 || group == 2 || group == 4 || group == 8);
}

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

cudaError_t launch_select_pages(const SelectParams &p, int dtype, int head_dim, int group, cudaStream_t s) {
    if (!sparse_supported(dtype, head_dim, group)) return cudaErrorNotSupported;
    if (dtype == PKV_BF16)
        return head_dim == 128 ? launch_select_g<bf16, 128>(p, group, s) : launch_select_g<bf16, 64>(p, group, s);
    return head_dim == 128 ? launch_select_g<float, 128>(p, group, s) : launch_select_g<float, 64>(p, group, s);
}

}  // namespace pkv
