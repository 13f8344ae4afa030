// pkv_select.cu -- which pages a sparse decode attends to (pkv_select_pages).
//
// The score of a page for a query q is the largest product that q can have with
// any key inside the page's bounds [lo, hi] (pkv_bounds.cu),
//   sum_c max(q_c lo_c, q_c hi_c) = q- . lo + q+ . hi   (q- <= 0 <= q+, q = q- + q+),
// maximised over the G query heads of the group.
//
// The selection must not depend on how a sum was rounded, so it is decided in
// two steps.  The score pass computes 32-bit scores s with |s - s*| <= e,
// where s* is the exact score and
//   e = kScoreEps * max_h sum_c |q[h, c]| * max |bound|,
// whose last two factors bound sum |terms|.  kScoreEps = 2^-16: a chain of four
// 16-term tensor-core products adds 17 numbers at a time, each off by 2^-23 of
// the largest at most when 24 bits are kept of what is aligned to it, 68 2^-23 <
// 2^-16.9 in all (fp32 units: 16 products and 3 additions a lane, less); the
// largest seen on this chip is 2^-20.6, on terms of very unlike sizes.  With T
// the 32-bit score of rank k, a page with s > T + 2e is in and one with s < T - 2e
// is out whatever the rounding was; the few in between are scored again in 64
// bits and ranked by (score, page).
#include <atomic>
#include <type_traits>

#include "pkv_launch.h"
#include "pkv_sparse.cuh"

namespace pkv {
namespace {

using bf16 = __nv_bfloat16;

constexpr float kScoreEps = 1.52587890625e-5f; // 2^-16
constexpr float kScoreTiny = 1e-35f;           // 256 products lost below the smallest normal number, doubled
constexpr int kBins = 1024;
constexpr int kUndecided = 256;          // scored in 64 bits from a list; more: by radix passes
constexpr int kMaxSplits = 8;            // CTAs of a cluster
constexpr int kStagedPages = 8192;       // pages whose scores fit a CTA's shared memory

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

// ---------------------------------------------------------------------------
// Scores of kScoreGroup = 16 pages of one entry and kv head, by a warp
// ---------------------------------------------------------------------------

// Tensor cores (bf16): the score is a product, [hi, lo] of 16 pages times
// [q+, q-] of the group's heads, so the pages are the rows and the heads the 8
// columns of m16n8k16.  A dot product may take its terms in any order, so lane
// (r, t) = (lane / 4, lane % 4) supplies the 16-byte chunks t, t + 4, ... of
// rows r and r + 8 (and of head r) straight from memory: four lanes read 64
// contiguous bytes, nothing is staged, and a warp has all of its 8 KB (D = 128)
// in flight at once.
template <typename T, int D, int G>
struct Scorer {
    static constexpr int kChunks = D / 8, kOwn = kChunks / 4;
    uint4 l0[kOwn], l1[kOwn], h0[kOwn], h1[kOwn], q[kOwn];

    // rows: n <= 8 rows of q, one for each column.
    __device__ __forceinline__ void load_q(const T *rows, int n) {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            q[j] = r < n ? reinterpret_cast<const uint4 *>(rows)[r * kChunks + t + 4 * j] : make_uint4(0, 0, 0, 0);
    }
    // Rows r and r + 8 of the group to load.  Bounds are read by plain loads: in a
    // step the kernel before this one writes them while this one is already
    // resident, and a load through the read-only path may be moved before the wait.
    const uint4 *r0, *r1;

    // The group to load next; phys: the physical page of its page lane % 16.
    __device__ __forceinline__ void aim(const SelectParams &p, int g, int phys) {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
        const uint4 *base = static_cast<const uint4 *>(p.page_bounds) + t;
        r0 = base + ((p.layer_page0 + __shfl_sync(0xffffffffu, phys, r)) * p.n_kv_heads + g) * 2 * kChunks;
        r1 = base + ((p.layer_page0 + __shfl_sync(0xffffffffu, phys, r + 8)) * p.n_kv_heads + g) * 2 * kChunks;
    }
    __device__ __forceinline__ void load_chunk(int j) {
        l0[j] = r0[4 * j];
        l1[j] = r1[4 * j];
        h0[j] = r0[kChunks + 4 * j];
        h1[j] = r1[kChunks + 4 * j];
    }
    __device__ __forceinline__ void load() {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) load_chunk(j);
    }
    // The largest |bound| of the group that is loaded (NaN kept).
    __device__ __forceinline__ float largest() const {
        uint4 most = h0[0], least = l0[0];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            widen_bounds<T>(least, most, l0[j], h0[j]);
            widen_bounds<T>(least, most, l1[j], h1[j]);
        }
        const uint32_t hi = max_word(max_word(most.x, most.y, T{}), max_word(most.z, most.w, T{}), T{});
        const uint32_t lo = min_word(min_word(least.x, least.y, T{}), min_word(least.z, least.w, T{}), T{});
        const float big = max_nan(max_nan(bf16lo(hi), bf16hi(hi)), -min_nan(bf16lo(lo), bf16hi(lo)));
        // non-negative numbers and NaN order like their bits
        return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big) & 0x7fffffffu));
    }
    // x: pages r (x[0], x[1]) and r + 8 of the group by columns 2t and 2t + 1.
    // kNext: each chunk is
    // loaded again, from the group aimed at, as soon as it is used, so that a
    // warp's loads never pause.
    template <bool kNext>
    __device__ __forceinline__ void products(float (&x)[4]) {
        x[0] = x[1] = x[2] = x[3] = 0.f;
        float y[4] = {}, z[4] = {}, w[4] = {};                    // four chains
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const uint4 qn = make_uint4(min_word(q[j].x, 0, T{}), min_word(q[j].y, 0, T{}), min_word(q[j].z, 0, T{}), min_word(q[j].w, 0, T{}));
            const uint4 qp = make_uint4(max_word(q[j].x, 0, T{}), max_word(q[j].y, 0, T{}), max_word(q[j].z, 0, T{}), max_word(q[j].w, 0, T{}));
            mma_bf16(x, l0[j].x, l1[j].x, l0[j].y, l1[j].y, qn.x, qn.y);
            mma_bf16(y, h0[j].x, h1[j].x, h0[j].y, h1[j].y, qp.x, qp.y);
            mma_bf16(z, l0[j].z, l1[j].z, l0[j].w, l1[j].w, qn.z, qn.w);
            mma_bf16(w, h0[j].z, h1[j].z, h0[j].w, h1[j].w, qp.z, qp.w);
            if (kNext) load_chunk(j);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (x[i] + z[i]) + (y[i] + w[i]);
    }
    // The score of page lane % 16 of the group for the first G columns.
    template <bool kNext>
    __device__ __forceinline__ float score() {
        const int lane = threadIdx.x & 31, t = lane & 3;
        float x[4];
        products<kNext>(x);
        float s0 = -INFINITY, s1 = -INFINITY;
        if (2 * t < G) {
            s0 = x[0];
            s1 = x[2];
        }
        if (2 * t + 1 < G) {
            s0 = max_nan(s0, x[1]);
            s1 = max_nan(s1, x[3]);
        }
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
            s0 = max_nan(s0, __shfl_xor_sync(0xffffffffu, s0, off));
            s1 = max_nan(s1, __shfl_xor_sync(0xffffffffu, s1, off));
        }
        s0 = __shfl_sync(0xffffffffu, s0, 4 * (lane & 7));
        s1 = __shfl_sync(0xffffffffu, s1, 4 * (lane & 7));
        return lane & 8 ? s1 : s0;
    }
    // The columns hold the G heads of each of kSets entries: put(entry, page of
    // the group, score), each from one lane.
    static constexpr int kSets = 8 / G;
    template <typename Put>
    __device__ __forceinline__ void score_sets(Put put) {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
        float x[4];
        products<false>(x);
        if constexpr (G == 1) {
            put(2 * t, r, x[0]);
            put(2 * t, r + 8, x[2]);
            put(2 * t + 1, r, x[1]);
            put(2 * t + 1, r + 8, x[3]);
        } else {
            float s0 = max_nan(x[0], x[1]), s1 = max_nan(x[2], x[3]);
#pragma unroll
            for (int off = 1; off < G / 2; off <<= 1) {
                s0 = max_nan(s0, __shfl_xor_sync(0xffffffffu, s0, off));
                s1 = max_nan(s1, __shfl_xor_sync(0xffffffffu, s1, off));
            }
            if (t % (G / 2) == 0) {
                put(2 * t / G, r, s0);
                put(2 * t / G, r + 8, s1);
            }
        }
    }
};

// CUDA cores (fp32): eight lanes to a page, four pages at a time, each lane
// the 16-byte chunks lane % 8, lane % 8 + 8, ... of the page's rows.
template <int D, int G>
struct Scorer<float, D, G> {
    static constexpr int kChunks = D / 4;
    const float *q;
    int page;                                // the physical page of page lane % 16 of the group

    __device__ __forceinline__ void load_q(const float *rows, int) { q = rows; }
    __device__ __forceinline__ void aim(const SelectParams &p, int g, int phys) {
        page = phys;
        base = static_cast<const uint4 *>(p.page_bounds) + (p.layer_page0 * p.n_kv_heads + g) * 2 * kChunks + (threadIdx.x & 7);
        step = static_cast<int64_t>(p.n_kv_heads) * 2 * kChunks;
    }
    __device__ __forceinline__ void load() { held = page; }
    const uint4 *base;
    int64_t step;
    int held;
    float big;
    // Of the group that was scored last.
    __device__ __forceinline__ float largest() const {
        return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big) & 0x7fffffffu));
    }
    template <bool kNext>
    __device__ __forceinline__ float score() {
        const int lane = threadIdx.x & 31, sub = lane & 7;
        float s = 0.f;
        big = 0.f;
#pragma unroll 1
        for (int i = 0; i < kScoreGroup; i += 4) {
            const uint4 *lo = base + __shfl_sync(0xffffffffu, held, i + (lane >> 3)) * step;
            float x[G];
#pragma unroll
            for (int h = 0; h < G; ++h) x[h] = 0.f;
#pragma unroll
            for (int c = 0; c < kChunks; c += 8) {
                float l[4], u[4];
                widen16(lo[c], l, float{});
                widen16(lo[kChunks + c], u, float{});
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    big = max_nan(big, max_nan(fabsf(l[e]), fabsf(u[e])));
#pragma unroll
                    for (int h = 0; h < G; ++h) {
                        const float qv = q[h * D + (c + sub) * 4 + e];
                        x[h] = fmaf(qv, qv >= 0.f ? u[e] : l[e], x[h]);
                    }
                }
            }
            float best = -INFINITY;
#pragma unroll
            for (int h = 0; h < G; ++h) {
#pragma unroll
                for (int off = 4; off >= 1; off >>= 1) x[h] += __shfl_xor_sync(0xffffffffu, x[h], off);
                best = max_nan(best, x[h]);
            }
            best = __shfl_sync(0xffffffffu, best, (lane & 3) * 8);
            if ((lane & 15) / 4 == i / 4) s = best;
        }
        if (kNext) load();
        return s;
    }
    static constexpr int kSets = 1;
    template <typename Put>
    __device__ __forceinline__ void score_sets(Put put) {
        const float s = score<false>();
        const int lane = threadIdx.x & 31;
        if (lane < 16) put(0, lane, s);
    }
};

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------

// Order-preserving integer keys; NaN above every number, -0 = +0.  kMarkIn is
// NaN's key.
constexpr uint32_t kMarkIn = 0xffffffffu;

__device__ __forceinline__ uint32_t key32(float s) {
    if (s != s) return kMarkIn;
    const uint32_t u = __float_as_uint(s + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unkey32(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// NT: threads of the selecting CTA.
template <int D, int G, int NT>
struct SelShared {
    static constexpr int kWarps = NT / 32;
    float q[G][D];
    int hist[kBins];
    unsigned long long warp_sum[kWarps];
    uint32_t lo[kWarps], hi[kWarps];
    uint32_t big[kMaxSplits * kWarps];    // the scoring warps' largest |bound|
    int bin, above;
    int und_page[kUndecided];
    unsigned long long und_key[kUndecided];
    uint32_t und_in[kUndecided / 32];
};

// Inclusive scan over the block of a whole number per thread.
template <int kWarps, typename N>
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
    N w = lane < kWarps ? static_cast<N>(warp_sum[lane]) : N(0);
#pragma unroll
    for (int off = 1; off < kWarps; off <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, kWarps - 1);
    const N before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return warp > 0 ? v + before : v;
}

// The bin (from the top) that holds rank `rank` (1-based) of the histogram:
// sh.bin, and sh.above = the count in higher bins.
template <int D, int G, int NT>
__device__ __forceinline__ void find_bin(SelShared<D, G, NT> &sh, int rank) {
    constexpr int kPer = kBins / NT;
    const int top = kBins - 1 - static_cast<int>(threadIdx.x) * kPer;   // this thread: top, top - 1, ...
    int c[kPer], own = 0, total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) own += c[k] = sh.hist[top - k];
    const int inc = block_scan<NT / 32>(sh.warp_sum, own, &total);
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

// Largest sum_c |q[h, c]| over the heads, every warp by itself.
template <int D, int G, int NT>
__device__ __forceinline__ float query_norm(const SelShared<D, G, NT> &sh) {
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

// Scores in 64-bit integers.  A product of two numbers of 24 bits is m 2^x with a
// whole m < 2^48.  A page's score for one query head is summed in units of
// 2^(X - 8), X the largest x of its own products: a term is below 2^56 units and
// the sum of 128 below 2^63.  Terms whose last bits fall below the unit lose them,
// less than 2^-54 of a product with X (a sum in fp64 is off by 2^-53 of each
// partial sum), the others are exact, and integer sums do not round, so the order
// of the terms does not matter.  The unit is the page's own: one taken from the
// largest bound of the entry would lose the whole score of pages beside one with
// an outlying channel.  The sum is then rounded to 53 bits, which makes it
// comparable with those of other units.  On integer units: fp64 arithmetic, and
// conversions to 64-bit integers with it, are so slow on this chip that a dozen
// pages took 4 to 9 us.

// An order-preserving key of v 2^x, rounded to the 53 bits of an fp64 number
// (ties to even); x within -1000 .. 900.  ~0 stands for NaN.
__device__ __forceinline__ unsigned long long key_of_sum(long long v, int x) {
    if (v == 0) return 1ull << 63;
    const unsigned long long size = v < 0 ? 0ull - static_cast<unsigned long long>(v) : static_cast<unsigned long long>(v);
    const int lz = __clzll(static_cast<long long>(size));
    const unsigned long long m = size << lz;                      // its first bit counts 2^(x - lz + 63)
    unsigned long long u = (static_cast<unsigned long long>(x - lz + 63 + 1023) << 52) + (m >> 11 & 0xfffffffffffffull);
    const unsigned rest = static_cast<unsigned>(m) & 0x7ffu;
    u += rest > 0x400u || (rest == 0x400u && (u & 1));
    return v < 0 ? ~(u | 1ull << 63) : u | 1ull << 63;
}

// The key of a page's score for one query head, by a warp whose lanes hold the
// page's bounds.  q and the bounds are finite; bf16 ones have 8 bits in place of
// 24, and products of 32 bits.
template <typename T, int D>
__device__ __forceinline__ unsigned long long integer_key(const float *q, const float (&l)[D / 32], const float (&u)[D / 32]) {
    constexpr int kLow = Elem<T>::bytes == 2 ? 16 : 0;            // bits of a significand that are 0
    using Product = typename std::conditional<kLow == 16, uint32_t, unsigned long long>::type;
    const int lane = threadIdx.x & 31;
    Product m[D / 32];                       // the product is m 2^(x - 300 + 2 kLow)
    int x[D / 32], most = 0;
    uint32_t sign[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const float qv = q[c * 32 + lane];
        const uint32_t a = __float_as_uint(qv), b = __float_as_uint(qv >= 0.f ? u[c] : l[c]);
        const uint32_t ea = a >> 23 & 255u, eb = b >> 23 & 255u;
        const uint32_t ma = (a & 0x7fffffu) | (ea ? 0x800000u : 0u), mb = (b & 0x7fffffu) | (eb ? 0x800000u : 0u);
        m[c] = static_cast<Product>(ma >> kLow) * (mb >> kLow);
        x[c] = static_cast<int>(max(ea, 1u) + max(eb, 1u));
        sign[c] = a ^ b;
        if (m[c]) most = max(most, x[c]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    long long s = 0;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {       // a product of 0 may have any x
        const long long units = static_cast<long long>((static_cast<unsigned long long>(m[c]) << (8 + 2 * kLow)) >> min(max(most - x[c], 0), 63));
        s += sign[c] >> 31 ? -units : units;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return key_of_sum(s, most - 308);
}

// Ranks the `n` <= kUndecided pages of sh.und_page by their integer scores and
// sets the bits of sh.und_in for the first `need` of them.  sh.und_key is 0 on
// entry, below every key.  A warp takes a page and as many of the heads, which
// share the loaded bounds, as keep all warps in work.
template <typename T, int D, int G, int NT, typename Phys>
__device__ __forceinline__ void rank_undecided(const SelectParams &p, SelShared<D, G, NT> &sh, int g, int n, int need, Phys phys) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int heads = 1;
    while (heads < G && n * (G / heads) > NT / 32) heads *= 2;
    for (int x = warp; x < n * (G / heads); x += NT / 32) {
        const int k = x / (G / heads), h0 = x % (G / heads) * heads;
        const T *lo = static_cast<const T *>(p.page_bounds) + ((p.layer_page0 + phys(sh.und_page[k])) * p.n_kv_heads + g) * 2 * D;
        float l[D / 32], u[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            l[c] = Elem<T>::to_f(lo[c * 32 + lane]);
            u[c] = Elem<T>::to_f(lo[D + c * 32 + lane]);
        }
        unsigned long long key = 0;
#pragma unroll 1
        for (int h = h0; h < h0 + heads; ++h) key = max(key, integer_key<T, D>(sh.q[h], l, u));
        if (lane == 0) atomicMax(&sh.und_key[k], key);
    }
    __syncthreads();
    bool in = false;
    if (tid < n) {
        const unsigned long long key = sh.und_key[tid];
        const int pg = sh.und_page[tid];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.und_key[j] > key || (sh.und_key[j] == key && sh.und_page[j] < pg);
        in = rank < need;
    }
    const unsigned bits = __ballot_sync(0xffffffffu, in);
    if (lane == 0 && warp < kUndecided / 32) sh.und_in[warp] = bits;
    __syncthreads();
}

// The key of a page's score over the group's heads, by a warp, for any q and
// bounds: with numbers that are not finite among them the score is infinite or
// NaN, as its products say.
template <typename T, int D, int G>
__device__ __forceinline__ unsigned long long any_key(const SelectParams &p, const float (&q)[G][D], int64_t bounds_row) {
    const int lane = threadIdx.x & 31;
    const T *lo = static_cast<const T *>(p.page_bounds) + bounds_row * 2 * D;
    float l[D / 32], u[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        l[c] = Elem<T>::to_f(lo[c * 32 + lane]);
        u[c] = Elem<T>::to_f(lo[D + c * 32 + lane]);
    }
    unsigned long long key = 0;
#pragma unroll 1
    for (int h = 0; h < G; ++h) {
        bool nan = false, up = false, down = false;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const float qv = q[h][c * 32 + lane], x = qv >= 0.f ? u[c] : l[c], y = qv * x;
            if (isfinite(qv) && isfinite(x)) continue;            // y may still overflow
            nan |= y != y;
            up |= y == INFINITY;
            down |= y == -INFINITY;
        }
        nan = __any_sync(0xffffffffu, nan);
        up = __any_sync(0xffffffffu, up);
        down = __any_sync(0xffffffffu, down);
        if (nan || (up && down)) return ~0ull;
        key = max(key, up ? 0xfffull << 52 : down ? ~(0xfffull << 52) : integer_key<T, D>(q[h], l, u));
    }
    return key;
}

// Many pages within rounding of the threshold (pages that are alike), or scores
// that are not finite: radix selection on 64-bit keys.  Each candidate's key is
// formed once and its upper half takes the place of its 32-bit score; the lower
// halves are formed again for those alone whose upper half is the threshold's,
// where these are too many.  Sets the keys of the `keep` best candidates to
// kMarkIn and those of the others to 0; candidates with scores above hi are in,
// those below lo out.  One request at 32K positions, pages of 16 with a NaN among
// them: 0.6 ms for the selection, all alike: 1.2 (13.4 with fp64 scores in each of
// nine passes).  Out of line, so that its registers are not the others'; p by
// reference wants a __grid_constant__ parameter, or every thread of the kernel
// begins with a copy in local memory (selection of 32 x 4K: 11.9 us, not 10.4).
template <typename T, int D, int G, int NT, typename Phys>
__device__ __noinline__ void select_by_radix(const SelectParams &p, SelShared<D, G, NT> &sh, int g, uint32_t *keys, int c0, int c1, uint32_t lo,
                                             uint32_t hi, int keep, Phys phys) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const auto key_of = [&](int page) { return any_key<T, D, G>(p, sh.q, (p.layer_page0 + phys(page)) * p.n_kv_heads + g); };
    for (int i = c0 + warp; i < c1; i += NT / 32) {
        const uint32_t k = keys[i];
        const uint32_t x = k > hi ? kMarkIn : k < lo ? 0u : static_cast<uint32_t>(key_of(i) >> 32);
        __syncwarp();
        if (lane == 0) keys[i] = x;
    }
    // the threshold, eight bits at a time; rank: how many of those equal to it are in
    int rank = keep;
    const auto narrow = [&](uint32_t &found, int shift, auto count) {
        for (int i = tid; i < kBins; i += NT) sh.hist[i] = 0;
        __syncthreads();
        count([&](uint32_t x) {
            if (shift == 24 || (x ^ found) >> (shift + 8) == 0) atomicAdd(&sh.hist[x >> shift & 255u], 1);
        });
        __syncthreads();
        find_bin(sh, rank);
        rank -= sh.above;
        found |= static_cast<uint32_t>(sh.bin) << shift;
    };
    uint32_t top = 0;
    for (int shift = 24; shift >= 0; shift -= 8)
        narrow(top, shift, [&](auto add) {
            for (int i = c0 + tid; i < c1; i += NT) add(keys[i]);
        });
    if (rank < sh.hist[sh.bin]) {            // the lower halves decide
        const auto each_low = [&](auto f) {
            for (int i = c0 + warp; i < c1; i += NT / 32)
                if (keys[i] == top) {
                    const uint32_t x = static_cast<uint32_t>(key_of(i));
                    if (lane == 0) f(x, i);
                }
        };
        __syncthreads();
        if (tid == 0) {
            sh.lo[0] = 0xffffffffu;
            sh.hi[0] = 0;
        }
        __syncthreads();
        each_low([&](uint32_t x, int) {
            atomicMin(&sh.lo[0], x);
            atomicMax(&sh.hi[0], x);
        });
        __syncthreads();
        if (sh.lo[0] != sh.hi[0]) {          // neither marked in nor out nor NaN: 0 < top < kMarkIn
            uint32_t low = 0;
            for (int shift = 24; shift >= 0; shift -= 8)
                narrow(low, shift, [&](auto add) { each_low([&](uint32_t x, int) { add(x); }); });
            each_low([&](uint32_t x, int i) {
                if (x != low) keys[i] = x > low ? kMarkIn : 0u;
            });
        }
    }
    __syncthreads();
    // those above the threshold are in, and the first `rank` that equal it
    const int per = (c1 - c0 + NT - 1) / NT, i0 = min(c1, c0 + tid * per), i1 = min(c1, i0 + per);
    int equal = 0, total;
    for (int i = i0; i < i1; ++i) equal += keys[i] == top;
    int before = block_scan<NT / 32>(sh.warp_sum, equal, &total) - equal;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = keys[i];
        keys[i] = k > top || (k == top && before++ < rank) ? kMarkIn : 0u;
    }
    __syncthreads();
}

// Selects from the keys of the entry's n > top_k pages (16-byte aligned, whole
// groups of kScoreGroup; shared or global memory) and writes sel.  Thread i
// holds a strip of consecutive pages; each pass (range, histogram, counts,
// output) ends in one block-wide scan, and what bounds it is their latency.
// big: the largest |bound| of this thread's share of the pages.  sh.q is set,
// sh.hist zero.  phys(page) is a page's physical page.
template <typename T, int D, int G, int NT, typename Phys>
__device__ __forceinline__ void select_from_keys(const SelectParams &p, SelShared<D, G, NT> &sh, int g, int n, uint32_t *keys, float big,
                                                   float norm, int32_t *sel, Phys phys) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int keep = p.top_k - p.n_first - p.n_last, c0 = p.n_first, c1 = n - p.n_last;   // candidates: pages c0 .. c1 - 1
    const int quads = ((n + 3) / 4 + NT - 1) / NT;                      // of pages, per thread
    const auto each = [&](auto f) {
        for (int c = 0; c < quads; ++c) {
            const int page = (tid * quads + c) * 4;
            if (page >= c1) break;
            const uint4 x = *reinterpret_cast<const uint4 *>(keys + page);
            const uint32_t k[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (page + i >= c0 && page + i < c1) f(k[i], page + i);
        }
    };
    uint32_t klo = 0xffffffffu, khi = 0;
    each([&](uint32_t k, int) {
        klo = min(klo, k);
        khi = max(khi, k);
    });
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    const uint32_t big_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(big) & 0x7fffffffu);
    if (lane == 0) {
        sh.lo[warp] = klo;
        sh.hi[warp] = khi;
        sh.big[warp] = big_bits;
    }
    __syncthreads();
    klo = __reduce_min_sync(0xffffffffu, sh.lo[lane % (NT / 32)]);
    khi = __reduce_max_sync(0xffffffffu, sh.hi[lane % (NT / 32)]);
    big = __uint_as_float(__reduce_max_sync(0xffffffffu, sh.big[lane % (NT / 32)]));
    if ((norm == 0.f || big == 0.f) && norm < INFINITY && big < INFINITY) {   // every score is 0: the lowest pages
        for (int i = tid; i < keep; i += NT) sel[c0 + i] = c0 + i;
        return;
    }
    const float slack = 2.f * kScoreEps * norm * big + kScoreTiny;   // 2e
    const bool finite = klo > key32(-INFINITY) && khi < key32(INFINITY) && slack < INFINITY;   // q, bounds and scores

    // the threshold's bin, the error bound on both sides included, as keys
    // [lo, hi], narrowed until few pages lie in it or a bin is one key
    uint32_t lo = 0, hi = 0xffffffffu;
    int above = 0, inside = c1 - c0;         // candidates above and in it
    int mine_above = 0, mine_inside = 0;     // of the threads before this one
    if (finite) {
        int rank = keep;
        for (;;) {
            const int shift = max(0, 32 - __clz(khi - klo) - 10);
            each([&](uint32_t k, int) {
                if (k >= klo && k <= khi) atomicAdd(&sh.hist[(k - klo) >> shift], 1);
            });
            __syncthreads();
            find_bin(sh, rank);
            rank -= sh.above;
            klo += static_cast<uint32_t>(sh.bin) << shift;
            khi = min(khi, klo + ((1u << shift) - 1u));
            lo = key32(unkey32(klo) - slack);
            hi = key32(unkey32(khi) + slack);
            unsigned long long both = 0, total;
            each([&](uint32_t k, int) { both += k > hi ? 1ull << 32 : k >= lo ? 1ull : 0ull; });
            const unsigned long long before = block_scan<NT / 32>(sh.warp_sum, both, &total) - both;
            above = static_cast<int>(total >> 32);
            inside = static_cast<int>(total);
            mine_above = static_cast<int>(before >> 32);
            mine_inside = static_cast<int>(before);
            if (inside <= kUndecided || shift == 0) break;
            for (int i = tid; i < kBins; i += NT) sh.hist[i] = 0;
            __syncthreads();
        }
    }
    const int need = keep - above;
    uint32_t least = lo;                     // keys from here on are in: the whole bin
    const bool listed = finite && need < inside && inside <= kUndecided;
    if (listed) {
        int k = mine_inside;
        each([&](uint32_t key, int page) {
            if (key >= lo && key <= hi) {
                sh.und_page[k] = page;
                sh.und_key[k++] = 0;
            }
        });
        __syncthreads();
        rank_undecided<T, D, G, NT>(p, sh, g, inside, need, phys);
    } else if (need < inside) {
        select_by_radix<T, D, G, NT>(p, sh, g, keys, c0, c1, lo, hi, keep, phys);
        least = kMarkIn;                     // those marked in
        int count = 0, total;
        each([&](uint32_t key, int) { count += key >= least; });
        mine_above = block_scan<NT / 32>(sh.warp_sum, count, &total) - count;
        mine_inside = 0;
    }
    // in ascending order; the list of undecided pages is ascending too
    int at = p.n_first + mine_above, k = mine_inside;
    if (listed) {
        for (int w = 0; w < k / 32; ++w) at += __popc(sh.und_in[w]);
        at += k % 32 ? __popc(sh.und_in[k / 32] & ((1u << (k % 32)) - 1u)) : 0;
    } else {
        at += k;
    }
    each([&](uint32_t key, int page) {
        if (key < least) return;
        if (listed && key <= hi) {
            const bool in = sh.und_in[k / 32] >> (k % 32) & 1;
            ++k;
            if (!in) return;
        }
        sel[at++] = page;
    });
}

// What every CTA of an entry and kv head begins with: q widened to sh.q, sh.hist
// zero, and, by `writer`, the count and the pages that need no score.  Returns
// the number of pages to score, 0 where nothing is left to select.
template <typename T, int D, int G, int NT>
__device__ __forceinline__ int begin_entry(const SelectParams &p, SelShared<D, G, NT> &sh, int g, int b, bool writer, int *row) {
    const int tid = threadIdx.x;
    for (int i = tid; i < G * D; i += NT)
        sh.q[i / D][i % D] = Elem<T>::to_f(static_cast<const T *>(p.q)[(static_cast<int64_t>(b) * p.n_heads + g * G) * D + i]);
    for (int i = tid; i < kBins; i += NT) sh.hist[i] = 0;
    const int n = entry_pages(p, b, row, writer && g == 0 && tid == 0);
    if (writer) {
        const int64_t unit = static_cast<int64_t>(b) * p.n_kv_heads + g;
        int32_t *sel = p.sel + unit * p.top_k;
        if (tid == 0) p.sel_counts[unit] = min(n, p.top_k);
        if (n <= p.top_k) {
            for (int i = tid; i < p.top_k; i += NT) sel[i] = i < n ? i : -1;
        } else {
            for (int i = tid; i < p.n_first; i += NT) sel[i] = i;
            for (int i = tid; i < p.n_last; i += NT) sel[p.top_k - p.n_last + i] = n - p.n_last + i;
        }
    }
    return n > p.top_k && p.top_k > p.n_first + p.n_last ? n : 0;
}

// Scores and selection in one launch: a cluster per (kv head, entry), whose
// warps share the groups of pages and put the scores' keys into the first CTA's
// shared memory; that CTA selects.
constexpr int kClusterThreads = 256;

template <typename T, int D, int G>
__global__ void __launch_bounds__(kClusterThreads, 2) select_cluster_kernel(const __grid_constant__ SelectParams p) {
    constexpr int NT = kClusterThreads, kWarps = NT / 32;
    __shared__ SelShared<D, G, NT> sh;
    extern __shared__ __align__(16) unsigned char staged[];
    uint32_t *keys = reinterpret_cast<uint32_t *>(staged);        // [page_cap]
    int *phys = reinterpret_cast<int *>(keys + p.page_cap);       // [page_cap]
    griddep_launch();
    const int rank = blockIdx.x, g = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int row;
    const int n = begin_entry<T, D, G, NT>(p, sh, g, b, rank == 0, &row);
    if (n == 0) {                                                 // for every CTA of the cluster
        if (p.pdl) griddep_wait();
        return;
    }
    if (p.splits > 1) cluster_arrive();                           // the first CTA's memory may be written once it runs
    const int groups = (n + kScoreGroup - 1) / kScoreGroup, step = p.splits * kWarps;
    int group = rank * kWarps + warp;
    const auto lookup = [&](int gr) { return gr < groups ? static_cast<int>(page_at(p, row, min(gr * kScoreGroup + (lane & 15), n - 1))) : 0; };
    Scorer<T, D, G> sc;
    int at = lookup(group);
    __syncthreads();
    if constexpr (Elem<T>::bytes == 4) sc.load_q(&sh.q[0][0], G);
    else sc.load_q(static_cast<const T *>(p.q) + (static_cast<int64_t>(b) * p.n_heads + g * G) * D, G);
    const float norm = rank == 0 ? query_norm(sh) : 0.f;
    if (p.pdl) griddep_wait();                                    // the bounds
    if (p.splits > 1) cluster_wait();
    float big = 0.f;
    if (group < groups) {
        sc.aim(p, g, at);
        sc.load();
    }
    while (group < groups) {
        const int next = lookup(group + step);
        constexpr bool kAfter = Elem<T>::bytes == 4;              // fp32 knows its largest bound after the scores
        if (!kAfter) big = max_nan(big, sc.largest());
        float s;
        if (group + step < groups) {
            sc.aim(p, g, next);
            s = sc.template score<true>();
        } else {
            s = sc.template score<false>();
        }
        if (kAfter) big = max_nan(big, sc.largest());
        if (lane < 16) {
            const int page = group * kScoreGroup + lane;
            st_cluster(cluster_addr(keys + page, 0), key32(s));
            st_cluster(cluster_addr(phys + page, 0), static_cast<uint32_t>(at));
        }
        at = next;
        group += step;
    }
    if (lane == 0) st_cluster(cluster_addr(&sh.big[rank * kWarps + warp], 0), __float_as_uint(big));
    if (p.splits > 1) cluster_sync();
    else __syncthreads();
    if (rank != 0) return;                                        // nobody reads its memory
    big = static_cast<int>(threadIdx.x) < p.splits * kWarps ? __uint_as_float(sh.big[threadIdx.x]) : 0.f;
    __syncthreads();                                              // sh.big is reused
    select_from_keys<T, D, G, NT>(p, sh, g, n, keys, big, norm, p.sel + (static_cast<int64_t>(b) * p.n_kv_heads + g) * p.top_k,
                                [&](int page) { return phys[page]; });
}

// The two kernels apart: scores to the workspace, then the selection.
//
// A warp scores one group of pages for p.entries consecutive entries, and reads
// the bounds again only where the request row changes: the queries of a prompt
// or a draft share them, and 8 / G of them share a product's columns.  Their q
// rows wait in shared memory.  256 queries of one prompt over 1024 pages: 110 us
// entry by entry, 52 with the bounds shared, 38 with the columns shared.
constexpr int kScoreWarps = 4;
constexpr int kMaxEntries = 16;
// Entries whose q rows take 32 KB at most.
template <typename T, int D, int G>
constexpr int max_entries() {
    return 32768 / (G * D * Elem<T>::bytes) < kMaxEntries ? 32768 / (G * D * Elem<T>::bytes) : kMaxEntries;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kScoreWarps * 32) score_pages_kernel(const SelectParams p) {
    constexpr int kEntries = max_entries<T, D, G>();              // p.entries at most
    __shared__ __align__(16) T q[kEntries][G * D];
    __shared__ int rows[kEntries], pages[kEntries];
    griddep_launch();
    const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b0 = static_cast<int>(blockIdx.z) * p.entries, entries = min(p.entries, p.batch - b0);
    if (tid < entries) pages[tid] = entry_pages(p, b0 + tid, &rows[tid], false);
    constexpr int kChunks = G * D * Elem<T>::bytes / 16;
    for (int i = tid; i < entries * kChunks; i += kScoreWarps * 32)
        reinterpret_cast<uint4 *>(q[i / kChunks])[i % kChunks] =
            __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + (static_cast<int64_t>(b0 + i / kChunks) * p.n_heads + g * G) * D) + i % kChunks);
    __syncthreads();
    if (p.pdl) griddep_wait();                                    // the bounds
    const int group = blockIdx.x * kScoreWarps + warp, first = group * kScoreGroup;
    Scorer<T, D, G> sc;
    int held_row = -1, held_pages = 0;       // what sc holds the bounds of
    float big = 0.f;
    for (int e = 0, count; e < entries; e += count) {
        // entries e .. e + count - 1 are of one request
        const int row = rows[e];
        int n = pages[e];
        for (count = 1; count < Scorer<T, D, G>::kSets && e + count < entries && rows[e + count] == row; ++count) n = max(n, pages[e + count]);
        if (n <= p.top_k || first >= n) continue;
        sc.load_q(q[e], count * G);
        constexpr bool kAfter = Elem<T>::bytes == 4;              // fp32 knows its largest bound after the scores
        if (row != held_row || (n > held_pages && first + kScoreGroup > held_pages)) {
            sc.aim(p, g, static_cast<int>(page_at(p, row, min(first + (lane & 15), n - 1))));
            sc.load();
            if (!kAfter) big = sc.largest();
            held_row = row;
            held_pages = n;
        }
        const int64_t unit = static_cast<int64_t>(b0 + e) * p.n_kv_heads + g;
        uint32_t *keys = p.keys + unit * p.page_cap + first;      // page_cap is whole groups
        const int64_t stride = static_cast<int64_t>(p.n_kv_heads) * p.page_cap;
        sc.score_sets([&](int set, int page, float s) {
            if (set < count) keys[set * stride + page] = key32(s);
        });
        if (kAfter) big = sc.largest();
        if (lane < count) p.group_max[(unit + static_cast<int64_t>(lane) * p.n_kv_heads) * (p.page_cap / kScoreGroup) + group] = big;
    }
}

template <typename T, int D, int G, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 6 : 2) select_pages_kernel(const __grid_constant__ SelectParams p) {
    __shared__ SelShared<D, G, NT> sh;
    extern __shared__ __align__(16) unsigned char staged[];
    griddep_launch();
    const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    int row;
    const int n = begin_entry<T, D, G, NT>(p, sh, g, b, true, &row);
    if (n == 0) {
        griddep_wait();
        return;
    }
    __syncthreads();
    const float norm = query_norm(sh);
    griddep_wait();                                               // the scores
    const int64_t unit = static_cast<int64_t>(b) * p.n_kv_heads + g;
    uint32_t *keys = p.keys + unit * p.page_cap;
    const float *gmax = p.group_max + unit * (p.page_cap / kScoreGroup);
    float big = 0.f;
    for (int i = tid; i < (n + kScoreGroup - 1) / kScoreGroup; i += NT) big = max_nan(big, gmax[i]);
    if (p.page_cap <= kStagedPages) {                             // read once
        uint4 *to = reinterpret_cast<uint4 *>(staged);
        for (int i = tid; i < (n + 3) / 4; i += NT) to[i] = reinterpret_cast<const uint4 *>(keys)[i];
        keys = reinterpret_cast<uint32_t *>(staged);
    }
    __syncthreads();
    select_from_keys<T, D, G, NT>(p, sh, g, n, keys, big, norm, p.sel + unit * p.top_k, [&](int page) { return page_at(p, row, page); });
}

template <typename K>
cudaError_t allow_smem(K kernel, std::atomic<uint64_t> &done, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    return cudaSuccess;
}

template <typename T, int D, int G>
cudaError_t launch_select(SelectParams p, cudaStream_t s) {
    if (p.entries > max_entries<T, D, G>()) p.entries = max_entries<T, D, G>();
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = attr;
    if (p.splits > 0) {
        cfg.blockDim = dim3(kClusterThreads);
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(select_cluster_kernel<T, D, G>, done, kStagedPages * 8);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(p.splits, p.n_kv_heads, p.batch);
        cfg.dynamicSmemBytes = static_cast<size_t>(p.keys ? p.page_cap : 0) * 8;
        cfg.numAttrs = p.pdl ? 1 : 0;
        if (p.splits > 1) {
            attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(p.splits);
            attr[cfg.numAttrs].val.clusterDim.y = 1;
            attr[cfg.numAttrs].val.clusterDim.z = 1;
            ++cfg.numAttrs;
        }
        return cudaLaunchKernelEx(&cfg, select_cluster_kernel<T, D, G>, p);
    }
    const int groups = p.page_cap / kScoreGroup;
    cfg.gridDim = dim3((groups + kScoreWarps - 1) / kScoreWarps, p.n_kv_heads, (p.batch + p.entries - 1) / p.entries);
    cfg.blockDim = dim3(kScoreWarps * 32);
    cfg.numAttrs = p.pdl ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, score_pages_kernel<T, D, G>, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.n_kv_heads, p.batch);
    cfg.dynamicSmemBytes = p.page_cap <= kStagedPages ? static_cast<size_t>(p.page_cap) * 4 : 0;
    cfg.numAttrs = 1;
    // More threads for a long list, more CTAs per SM for short ones.  Measured with
    // 512 threads against 256: 16 x 128K positions in pages of 32 42 us against 55,
    // one x 128K in pages of 16 18 against 52, 64 x 64K 206 against 214; 256 queries
    // over 1024 pages 165 against 147, 256 x 4K 93 against 73.  (Between them 512
    // measured a little better for 16 x 32K, 38 against 42.)
    cfg.blockDim = dim3(p.page_cap > 2048 ? 512 : 256);
    return p.page_cap > 2048 ? cudaLaunchKernelEx(&cfg, select_pages_kernel<T, D, G, 512>, p)
                             : cudaLaunchKernelEx(&cfg, select_pages_kernel<T, D, G, 256>, p);
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

// One launch (a cluster per entry and kv head) while the resident warps, 16 per
// SM, have two groups of pages each at most: what counts is then the launches
// and the latency of the passes.  Two launches where the bounds are many: the
// cluster's CTAs would hold their SMs while one of them selects, and the queries
// of one request would not share bounds.  Measured, GPU time of the call in one
// launch against two: selection for 32 x 4K positions 10.4 us against 13.6, a
// step of one request at 32K 17.3 against 19.2, of 16 x 4K 22.6 against 26.3;
// selection for 16 x 128K in pages of 32 47.8 against 42.3, a step of 256 queries
// of one prompt 199 against 147.  Batches of contexts that share nothing lie
// between: 64 x 4K 20 against 22, 16 x 32K 35 against 42, 64 x 32K 103 against 112.
void select_plan(SelectParams *p, int sms) {
    const int64_t units = static_cast<int64_t>(p->batch) * p->n_kv_heads, groups = p->page_cap / kScoreGroup;
    const int64_t warps = 16LL * sms;
    p->splits = 0;
    p->entries = 1;
    if (p->page_cap <= kStagedPages && units * groups <= 2 * warps) {
        int64_t splits = 2LL * sms / units;
        const int64_t most = (groups + kClusterThreads / 32 - 1) / (kClusterThreads / 32);
        if (splits > most) splits = most;
        p->splits = static_cast<int>(splits < 1 ? 1 : splits > kMaxSplits ? kMaxSplits : splits);
        return;
    }
    // as many entries per warp as leave four rounds of resident warps
    const int64_t entries = units * groups / (4 * warps);
    p->entries = static_cast<int>(entries < 1 ? 1 : entries > kMaxEntries ? kMaxEntries : entries);
}

cudaError_t launch_select_pages(const SelectParams &p, int dtype, int head_dim, int group, cudaStream_t s) {
    if (!sparse_supported(dtype, head_dim, group)) return cudaErrorNotSupported;
    if (dtype == PKV_BF16)
        return head_dim == 128 ? launch_select_g<bf16, 128>(p, group, s) : launch_select_g<bf16, 64>(p, group, s);
    return head_dim == 128 ? launch_select_g<float, 128>(p, group, s) : launch_select_g<float, 64>(p, group, s);
}

}  // namespace pkv
