// pkv_selected.cu -- decode attention over selected pages
// (pkv_paged_decode_selected): for each entry and kv head the pages of a list,
// read through the page table.
//
// Work split: one thread-block cluster per (entry, kv head).  Its CTAs share
// the list's positions in blocks of kBlk, each warp takes blocks of its CTA's
// run with an online softmax of its own (base 2), the warps' partials meet in
// shared memory and the CTAs' partials in distributed shared memory, so there
// is one launch and no workspace.  A list is bounded by top_k pages, and the
// host picks the cluster size so that all SMs have work.
#include <atomic>

#include "pkv_launch.h"
#include "pkv_sparse.cuh"

namespace pkv {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kBlk = 16;              // positions per block
constexpr int kStagePages = 512;      // list entries resolved to slots at a time
constexpr int kMaxSplits = 8;         // CTAs per cluster (the portable limit)

__device__ __forceinline__ float weight(float m, float top) { return m == -INFINITY ? 0.f : fast_exp2(m - top); }

// One listed page: its first slot and its first position (-1: not to be read).
struct Run {
    int slot, pos;
};

// Partial softmax states of a CTA's kParts parts of kHeads heads.
template <int kParts, int kHeads, int D>
struct Partials {
    float m[kParts][kHeads];
    float l[kParts][kHeads];
    float scale[kParts][kHeads];         // of the parts towards their common maximum
    float top[kHeads], sum[kHeads];      // the CTA's maximum and denominator
    alignas(16) float o[kParts][kHeads][D];
};

template <typename T>
__device__ __forceinline__ void store4(T *to, const float4 &x) {
    if constexpr (Elem<T>::bytes == 4) {
        *reinterpret_cast<float4 *>(to) = x;
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2 *>(to) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

// Joins the parts of every CTA of the cluster and writes o.  A CTA alone writes
// its sums; in a cluster part 0 becomes the CTA's own partial, and CTA r sums
// its share of the outputs over all CTAs.
template <typename T, int kParts, int kHeads, int D, int kThreads>
__device__ __forceinline__ void join(Partials<kParts, kHeads, D> &sh, T *out, int rank, int splits) {
    const int tid = threadIdx.x;
    constexpr int kOut = kHeads * D;
    __syncthreads();
    if (tid < kHeads) {
        float top = sh.m[0][tid], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kParts; ++w) top = fmaxf(top, sh.m[w][tid]);
#pragma unroll
        for (int w = 0; w < kParts; ++w) {
            const float f = weight(sh.m[w][tid], top);
            sh.scale[w][tid] = f;
            sum = fmaf(sh.l[w][tid], f, sum);
        }
        sh.top[tid] = top;
        sh.sum[tid] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (kOut + kThreads * 4 - 1) / (kThreads * 4); ++i) {
        const int e = (tid + i * kThreads) * 4, h = e / D, c = e % D;
        if (e >= kOut) break;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kParts; ++w) {
            const float f = sh.scale[w][h];
            const float4 x = *reinterpret_cast<const float4 *>(&sh.o[w][h][c]);
            acc.x = fmaf(f, x.x, acc.x);
            acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z);
            acc.w = fmaf(f, x.w, acc.w);
        }
        if (splits == 1) {
            const float l = sh.sum[h], inv = l == 0.f ? 0.f : 1.f / l;
            store4(out + e, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        } else {
            *reinterpret_cast<float4 *>(&sh.o[0][h][c]) = acc;    // read by this thread alone so far
        }
    }
    if (splits == 1) return;
    cluster_sync();
    const int e1 = kOut * (rank + 1) / splits;
    for (int e = kOut * rank / splits + tid; e < e1; e += kThreads) {
        const int h = e / D, c = e % D;
        float mr[kMaxSplits], lr[kMaxSplits], xr[kMaxSplits], all = -INFINITY, l = 0.f, x = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) {           // all in flight together
            const bool there = r < splits;
            mr[r] = there ? ld_cluster(cluster_addr(&sh.top[h], r)) : -INFINITY;
            lr[r] = there ? ld_cluster(cluster_addr(&sh.sum[h], r)) : 0.f;
            xr[r] = there ? ld_cluster(cluster_addr(&sh.o[0][h][c], r)) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) all = fmaxf(all, mr[r]);
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) {
            const float f = weight(mr[r], all);
            l = fmaf(f, lr[r], l);
            x = fmaf(f, xr[r], x);
        }
        out[e] = Elem<T>::from_f(l == 0.f ? 0.f : x / l);
    }
    cluster_sync();                      // no CTA leaves while its memory is read
}

// What a CTA attends to: blocks [t0, t1) of the list's flattened positions.  The
// lists are read by plain loads: in a step the selection writes them while this
// kernel is already resident.
struct Share {
    int row, len, n_pages, t0, t1;
};

__device__ __forceinline__ Share cta_share(const SelectedParams &p, int g, int b, int rank, bool report) {
    Share s;
    s.row = __ldg(p.req_pool_indices + b);
    s.len = __ldg(p.seq_lens + b);
    int count = p.sel_counts[static_cast<int64_t>(b) * p.n_kv_heads + g];
    if (static_cast<unsigned>(s.row) >= static_cast<unsigned>(p.num_reqs)) {
        if (report) record_error(p.err, s.row);
        s.row = s.len = count = 0;
    }
    if (s.len < 0 || s.len > p.max_len) {
        if (report) record_error(p.err, s.len);
        s.len = s.len < 0 ? 0 : p.max_len;
    }
    if (count < 0 || count > p.top_k) {
        if (report) record_error(p.err, count);
        count = count < 0 ? 0 : p.top_k;
    }
    s.n_pages = s.len / p.page_size + (s.len % p.page_size != 0);
    // top_k * page_size fits 31 bits (checked on the host)
    const int total = count * p.page_size;
    const int blocks = total / kBlk + (total % kBlk != 0);
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / p.splits);
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / p.splits);
    s.t0 = b0 * kBlk;
    s.t1 = min(total, b1 * kBlk);
    return s;
}

// The list entry that this thread resolves first if the list is full: it is
// loaded beside the count and not after it.
struct Guess {
    int first, page;
};
__device__ __forceinline__ Guess guess_entry(const SelectedParams &p, const int32_t *sel, int rank) {
    const int blocks = (p.top_k * p.page_size + kBlk - 1) / kBlk;
    Guess x;
    x.first = static_cast<int>(static_cast<int64_t>(blocks) * rank / p.splits) * kBlk / p.page_size;
    const int i = x.first + static_cast<int>(threadIdx.x);
    x.page = i < p.top_k ? sel[i] : 0;
    return x;
}

// Resolves list entries [i0, i1) to slots.
template <int kThreads>
__device__ __forceinline__ void stage_runs(const SelectedParams &p, const Share &s, const int32_t *sel, const Guess &guess, int i0, int i1, Run *runs) {
    for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += kThreads) {
        const int page = i == guess.first + static_cast<int>(threadIdx.x) ? guess.page : sel[i];
        Run r{0, -1};
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(s.n_pages)) {
            record_error(p.err, page);
        } else {
            int phys = __ldg(p.req_to_page + static_cast<int64_t>(s.row) * p.max_pages + page);
            if (static_cast<unsigned>(phys) >= static_cast<unsigned long long>(p.n_pages)) {
                record_error(p.err, phys);
                phys = 0;
            }
            r.slot = phys * p.page_size;
            r.pos = page * p.page_size;
        }
        runs[i - i0] = r;
    }
}

// ---------------------------------------------------------------------------
// CUDA cores (fp32): eight lanes to a position, kHeads query heads of the kv head
// ---------------------------------------------------------------------------

constexpr int kSimtWarps = 4;
constexpr int kSimtThreads = kSimtWarps * 32;

template <int D, int kHeads>
__global__ void __launch_bounds__(kSimtThreads) selected_simt_kernel(const SelectedParams p) {
    using T = float;
    constexpr int kElems = 16 / Elem<T>::bytes;
    constexpr int kChunks = D / kElems;
    constexpr int kOwn = kChunks / 8;                // 16-byte chunks of a row per lane
    __shared__ Partials<kSimtWarps, kHeads, D> sh;
    __shared__ float q[kHeads][D];
    __shared__ Run runs[kStagePages];
    griddep_launch();
    const int group = p.n_heads / p.n_kv_heads;
    const int rank = blockIdx.x, h0 = blockIdx.y * kHeads, g = h0 / group, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & 7;
    const int64_t out0 = (static_cast<int64_t>(b) * p.n_heads + h0) * D;
    for (int i = tid; i < kHeads * D; i += kSimtThreads)
        q[i / D][i % D] = Elem<T>::to_f(static_cast<const T *>(p.q)[out0 + i]) * p.scale_log2;
    if (p.pdl) griddep_wait();
    const int32_t *sel = p.sel + (static_cast<int64_t>(b) * p.n_kv_heads + g) * p.top_k;
    const Guess guess = guess_entry(p, sel, rank);
    const Share s = cta_share(p, g, b, rank, rank == 0 && h0 % group == 0 && tid == 0);

    float m[kHeads], l[kHeads], o[kHeads][kOwn * kElems];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int c = 0; c < kOwn * kElems; ++c) o[h][c] = 0.f;
    }
    const int i_end = s.t1 > s.t0 ? (s.t1 - 1) / p.page_size + 1 : 0;
    for (int i0 = s.t0 / p.page_size; i0 < i_end; i0 += kStagePages) {
        const int i1 = min(i_end, i0 + kStagePages);
        __syncthreads();
        stage_runs<kSimtThreads>(p, s, sel, guess, i0, i1, runs);
        __syncthreads();
        const int from = max(s.t0, i0 * p.page_size);
        const int to = static_cast<int>(min(static_cast<int64_t>(s.t1), static_cast<int64_t>(i1) * p.page_size));
        for (int t = from + warp * 4; t < to; t += kSimtWarps * 4) {     // warp-uniform
            const int tt = min(t + (lane >> 3), to - 1);
            const int i = tt / p.page_size, off = tt - i * p.page_size;
            const Run r = runs[i - i0];
            const bool seen = t + (lane >> 3) < to && r.pos >= 0 &&
                              static_cast<unsigned>(r.pos) + off < static_cast<unsigned>(s.len);
            const int64_t at = ((p.layer_row0 + r.slot + (seen ? off : 0)) * p.n_kv_heads + g) * kChunks + sub;
            const uint4 *kr = static_cast<const uint4 *>(p.k_buffer) + at;
            const uint4 *vr = static_cast<const uint4 *>(p.v_buffer) + at;
            float w[kHeads];
#pragma unroll
            for (int h = 0; h < kHeads; ++h) w[h] = 0.f;
            if (seen) {
#pragma unroll
                for (int c = 0; c < kOwn; ++c) {
                    float x[kElems];
                    load_widen<T, kElems>(reinterpret_cast<const T *>(kr + c * 8), x);
#pragma unroll
                    for (int h = 0; h < kHeads; ++h)
#pragma unroll
                        for (int e = 0; e < kElems; ++e) w[h] = fmaf(q[h][(c * 8 + sub) * kElems + e], x[e], w[h]);
                }
            }
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
#pragma unroll
                for (int x = 4; x >= 1; x >>= 1) w[h] += __shfl_xor_sync(0xffffffffu, w[h], x);
                if (!seen) w[h] = -INFINITY;
            }
            if (seen) {
                float x[kOwn * kElems];
#pragma unroll
                for (int c = 0; c < kOwn; ++c) {
                    float y[kElems];
                    load_widen<T, kElems>(reinterpret_cast<const T *>(vr + c * 8), y);
#pragma unroll
                    for (int e = 0; e < kElems; ++e) x[c * kElems + e] = y[e];
                }
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    const float top = fmaxf(m[h], w[h]);
                    const float f = weight(m[h], top), pr = weight(w[h], top);
                    m[h] = top;
                    l[h] = fmaf(l[h], f, pr);
#pragma unroll
                    for (int c = 0; c < kOwn * kElems; ++c) o[h][c] = fmaf(o[h][c], f, pr * x[c]);
                }
            }
        }
    }
    // the four positions of a warp, then the warps
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        float top = m[h];
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float f = weight(m[h], top);
        float sum = l[h] * f;
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (lane == 0) {
            sh.m[warp][h] = top;
            sh.l[warp][h] = sum;
        }
#pragma unroll
        for (int c = 0; c < kOwn; ++c)
#pragma unroll
            for (int e = 0; e < kElems; ++e) {
                float x = o[h][c * kElems + e] * f;
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (lane < 8) sh.o[warp][h][(c * 8 + sub) * kElems + e] = x;
            }
    }
    join<T, kSimtWarps, kHeads, D, kSimtThreads>(sh, static_cast<T *>(p.o) + out0, rank, p.splits);
}

// ---------------------------------------------------------------------------
// Tensor cores (bf16)
// ---------------------------------------------------------------------------

constexpr int kMmaWarps = 4;
constexpr float kRaise = 8.f;
constexpr int kMmaThreads = kMmaWarps * 32;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// The slot of position lane % 16 of the block at `at`, -1 where there is none.
__device__ __forceinline__ int slot_at(int at, int to, int i0, const Run *runs, const SelectedParams &p, int len) {
    const int x = at + static_cast<int>(threadIdx.x & 15);
    if (x >= to) return -1;
    const int i = p.page_shift >= 0 ? x >> p.page_shift : x / p.page_size, off = x - i * p.page_size;
    const Run run = runs[i - i0];
    return run.pos >= 0 && static_cast<unsigned>(run.pos) + off < static_cast<unsigned>(len) ? run.slot + off : -1;
}

// 2^x to 2^-22 of the value, 0 for -inf.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ void cp_async16_at(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// Shared memory of a CTA: each warp's ring of kRing half blocks (16 rows of K or
// of V), whose space the partials take over in the end, and the staged runs.
template <int D, int G>
struct MmaShared {
    static constexpr int kRing = 3;
    static constexpr int kRows = kBlk * D;                        // elements of a half block
    union {
        bf16 ring[kMmaWarps][kRing][kRows];
        Partials<kMmaWarps, G, D> parts;
    };
    Run runs[kStagePages];
};

// Where chunk c of a half block's row stands, so that lanes that read together
// hit different banks: two rows by four chunks of K, eight rows by a chunk of V.
__device__ __forceinline__ int swizzle_k(int row, int c) { return c ^ (row & 1) << 2; }
__device__ __forceinline__ int swizzle_v(int row, int c) { return c ^ (row & 7); }

// Four 8 x 8 blocks of 16-bit elements, transposed: lane l gives the address of
// row l % 8 of block l / 8.
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

// Bound by the bytes of the selected rows: 64 requests x 2048 positions of 8 kv
// heads (537 MB, gathered in runs of 256 bytes) take 89 us, 6.0 TB/s, 0.89 of the
// copy rate; 256 queries of one prompt, whose 1.07 GB come from L2, take 85 us
// and are bound by the waits of dependent instructions in each warp's one chain
// (0.45 of the issue slots; 104 with V transposed by byte permutations and a
// rescaling whenever the maximum moved, 95 with the join's weights formed for
// every output); one request is bound by the chain list -> page table -> rows ->
// join (7 us).
//
// A warp takes a block of 16 positions at a time.  K and V rows come by cp.async
// into the warp's own ring, two half blocks ahead of the one in use, so there is
// no barrier in the loop, and 16 warps keep 128 KB in flight per SM (rows loaded
// straight into registers, a block at a time: 114 us).  With lane
// (r, t) = (lane / 4, lane % 4):
//   S[8 heads x 16]   = Q K^T: a dot product may take its terms in any order,
//     so lane (r, t) takes the 16-byte chunks t, t + 4, ... of the K rows r and
//     r + 8 (and of head r's q) and feeds them as the columns 2t, 2t + 1, 2t +
//     8, 2t + 9 of successive k steps;
//   O^T[D x 8 heads] += V^T P^T: P of positions 2t, 2t + 1, 2t + 8, 2t + 9 and
//     head r is where S left it, and ldmatrix transposes V.
// The weights are relative to a reference m that is raised only when a score
// passes it by kRaise (2^8): sums and outputs keep their 24 bits, and most blocks
// need neither the maximum across lanes nor a rescaling.
// P goes in as two bf16 parts (hi + lo, 16 bits together): one part alone would
// add an error of the size of the output's own rounding.  With two, 0.25 % of the
// outputs round to the bf16 next to that of the 64-bit value, with three (24
// bits) 0.1 %, with fp32 sums in torch 0.06 %; the error from the 64-bit value is
// the same to six digits, and the third part costs 1 to 5 % of the time.  (A V
// that is infinite may give NaN, 0 times infinity, and not infinity.)
template <int D, int G>
__global__ void __launch_bounds__(kMmaThreads, 4) selected_mma_kernel(const SelectedParams p) {
    using Sh = MmaShared<D, G>;
    constexpr int kChunks = D / 8, kOwn = kChunks / 4, kRing = Sh::kRing;
    extern __shared__ __align__(128) unsigned char smem[];
    Sh &sh = *reinterpret_cast<Sh *>(smem);
    griddep_launch();
    const int rank = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
    const int64_t out0 = (static_cast<int64_t>(b) * p.n_heads + g * G) * D;
    uint4 q[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        q[j] = r < G ? __ldg(static_cast<const uint4 *>(p.q) + out0 / 8 + r * kChunks + t + 4 * j) : make_uint4(0, 0, 0, 0);
    if (p.pdl) griddep_wait();
    const int32_t *sel = p.sel + (static_cast<int64_t>(b) * p.n_kv_heads + g) * p.top_k;
    const Guess guess = guess_entry(p, sel, rank);
    const Share s = cta_share(p, g, b, rank, rank == 0 && threadIdx.x == 0);

    float m = -INFINITY, l = 0.f;            // head r; l over this lane's positions
    float o[D / 16][4];                      // channels 16 i + r and 16 i + r + 8, heads 2t, 2t + 1 of each
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    // A half block to ring place `to`: kRowLanes lanes to a row.  An unseen
    // position's K is slot 0's (its score is masked), its V zeros.
    constexpr int kRowLanes = kChunks, kRowsPer = 32 / kRowLanes, kRowBytes = D * 2, kPlaceBytes = Sh::kRows * 2;
    const uint32_t ring = smem_u32(sh.ring[warp][0]);
    const int64_t lane0 = (p.layer_row0 * p.n_kv_heads + g) * kRowBytes + lane % kRowLanes * 16;
    const char *kp = static_cast<const char *>(p.k_buffer) + lane0, *vp = static_cast<const char *>(p.v_buffer) + lane0;
    const uint32_t slot_bytes = static_cast<uint32_t>(p.n_kv_heads) * kRowBytes;
    constexpr int kFills = 8 / kRowsPer;     // places of a lane among eight rows; eight rows on the same again
    uint32_t put_k[kFills], put_v[kFills];
#pragma unroll
    for (int i = 0; i < kFills; ++i) {
        const int row = i * kRowsPer + lane / kRowLanes;
        put_k[i] = row * kRowBytes + swizzle_k(row, lane % kRowLanes) * 16;
        put_v[i] = row * kRowBytes + swizzle_v(row, lane % kRowLanes) * 16;
    }
    const auto fetch_k = [&](int slot, int to) {
        const int safe = max(slot, 0);
        const uint32_t place = ring + to * kPlaceBytes;
#pragma unroll
        for (int i = 0; i < kBlk / kRowsPer; ++i) {
            const uint32_t from = __shfl_sync(0xffffffffu, safe, i * kRowsPer + lane / kRowLanes);
            cp_async16_at(place + put_k[i % kFills] + i / kFills * 8 * kRowBytes, kp + static_cast<uint64_t>(from) * slot_bytes, 16);
        }
        cp_async_commit();
    };
    const auto fetch_v = [&](int slot, int to) {
        const uint32_t place = ring + to * kPlaceBytes;
        if (__all_sync(0xffffffffu, slot >= 0)) {
#pragma unroll
            for (int i = 0; i < kBlk / kRowsPer; ++i) {
                const uint32_t from = __shfl_sync(0xffffffffu, slot, i * kRowsPer + lane / kRowLanes);
                cp_async16_at(place + put_v[i % kFills] + i / kFills * 8 * kRowBytes, vp + static_cast<uint64_t>(from) * slot_bytes, 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kBlk / kRowsPer; ++i) {
                const int from = __shfl_sync(0xffffffffu, slot, i * kRowsPer + lane / kRowLanes);
                cp_async16_at(place + put_v[i % kFills] + i / kFills * 8 * kRowBytes,
                              vp + static_cast<uint64_t>(static_cast<uint32_t>(max(from, 0))) * slot_bytes, from >= 0 ? 16 : 0);
            }
        }
        cp_async_commit();
    };
    // Places of this lane's chunks: K row r, chunks t + 4 j for j even and odd
    // (128 bytes on for each j / 2, eight rows on for row r + 8); V row lane % 8
    // (+ 8 for the upper half of the lanes), chunk lane / 8 % 2: 2 i + that chunk
    // is 32 i bytes away by exclusive or.
    const uint32_t k_even = ring + r * kRowBytes + swizzle_k(r, t) * 16, k_odd = ring + r * kRowBytes + swizzle_k(r, t + 4) * 16;
    const int v_row = (lane & 7) + (lane >> 4) * 8;
    const uint32_t v_at = ring + v_row * kRowBytes + swizzle_v(v_row, lane >> 3 & 1) * 16;

    const int i_end = s.t1 > s.t0 ? (s.t1 - 1) / p.page_size + 1 : 0;
    for (int i0 = s.t0 / p.page_size; i0 < i_end; i0 += kStagePages) {
        const int i1 = min(i_end, i0 + kStagePages);
        __syncthreads();
        stage_runs<kMmaThreads>(p, s, sel, guess, i0, i1, sh.runs);
        __syncthreads();
        const int from = max(s.t0, i0 * p.page_size);
        const int to = static_cast<int>(min(static_cast<int64_t>(s.t1), static_cast<int64_t>(i1) * p.page_size));
        int at = from + warp * kBlk, x = 0;                       // x: ring place of the half block in use
        if (at >= to) continue;
        int slot = slot_at(at, to, i0, sh.runs, p, s.len);
        fetch_k(slot, 0);
        fetch_v(slot, 1);
        const auto after = [&](int place, int by) { return place + by < kRing ? place + by : place + by - kRing; };
        while (at < to) {
            const int next = at + kMmaWarps * kBlk;
            const int next_slot = slot_at(next, to, i0, sh.runs, p, s.len);
            if (next < to) fetch_k(next_slot, after(x, 2));
            else cp_async_commit();
            const unsigned unseen = ~__ballot_sync(0xffffffffu, slot >= 0);
            cp_async_wait<2>();
            __syncwarp();
            float w[2][4] = {};
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 k = lds16((j & 1 ? k_odd : k_even) + x * kPlaceBytes + (j / 2) * 128 + i * 8 * kRowBytes);
                    mma_bf16(w[i], q[j].x, 0, q[j].y, 0, k.x, k.y);
                    mma_bf16(w[i], q[j].z, 0, q[j].w, 0, k.z, k.w);
                }
            // head r, positions 2t, 2t + 1, 2t + 8, 2t + 9
            float pr[4] = {w[0][0] * p.scale_log2, w[0][1] * p.scale_log2, w[1][0] * p.scale_log2, w[1][1] * p.scale_log2};
            if (unseen) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (unseen >> (2 * t + (i & 1) + 8 * (i >> 1)) & 1) pr[i] = -INFINITY;
            }
            float top = fmaxf(fmaxf(pr[0], pr[1]), fmaxf(pr[2], pr[3]));
            if (__any_sync(0xffffffffu, top > m + kRaise)) {      // m = -inf: as soon as something is seen
                top = fmaxf(top, m);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float f = weight(m, top);
                m = top;
                l *= f;
                const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    o[i][0] *= f0;
                    o[i][1] *= f1;
                    o[i][2] *= f0;
                    o[i][3] *= f1;
                }
            }
            const float zero = m == -INFINITY ? 0.f : m;          // nothing seen yet: weights exp2(-inf) = 0
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pr[i] = exp2_approx(pr[i] - zero);
                l += pr[i];
            }
            const uint32_t hi0 = pack_bf16(pr[0], pr[1]), hi1 = pack_bf16(pr[2], pr[3]);
            const uint32_t lo0 = pack_bf16(pr[0] - bf16lo(hi0), pr[1] - bf16hi(hi0));
            const uint32_t lo1 = pack_bf16(pr[2] - bf16lo(hi1), pr[3] - bf16hi(hi1));
            __syncwarp();                                         // every lane has read the K rows
            if (next < to) fetch_v(next_slot, x);
            else cp_async_commit();
            x = after(x, 1);
            cp_async_wait<2>();
            __syncwarp();
            const uint32_t v_place = v_at + x * kPlaceBytes;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t v[4];
                ldmatrix_t(v, (v_place ^ (i % 4) * 32) + i / 4 * 128);
                mma_bf16(o[i], v[0], v[1], v[2], v[3], hi0, hi1);
                mma_bf16(o[i], v[0], v[1], v[2], v[3], lo0, lo1);
            }
            __syncwarp();                                         // every lane has read the V rows
            x = after(x, 1);
            at = next;
            slot = next_slot;
        }
    }
    cp_async_wait<0>();
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    __syncthreads();                                              // the rings become the partials
    if (t == 0 && r < G) {
        sh.parts.m[warp][r] = m;
        sh.parts.l[warp][r] = l;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (2 * t + (e & 1) < G) sh.parts.o[warp][2 * t + (e & 1)][16 * i + r + (e >> 1) * 8] = o[i][e];
    join<bf16, kMmaWarps, G, D, kMmaThreads>(sh.parts, static_cast<bf16 *>(p.o) + out0, rank, p.splits);
}

template <typename K>
cudaError_t launch_cluster(K kernel, dim3 grid, int threads, size_t smem, const SelectedParams &p, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (p.splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(p.splits);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (p.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int G>
cudaError_t run_mma(const SelectedParams &p, cudaStream_t s) {
    constexpr size_t smem = sizeof(MmaShared<D, G>);
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        e = cudaFuncSetAttribute(selected_mma_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        attr_done.fetch_or(bit);
    }
    return launch_cluster(selected_mma_kernel<D, G>, dim3(p.splits, p.n_kv_heads, p.batch), kMmaThreads, smem, p, s);
}

template <int D>
cudaError_t run_mma_g(const SelectedParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return run_mma<D, 1>(p, s);
        case 2: return run_mma<D, 2>(p, s);
        case 4: return run_mma<D, 4>(p, s);
        default: return run_mma<D, 8>(p, s);
    }
}

template <int D, int kHeads>
cudaError_t run_simt(const SelectedParams &p, cudaStream_t s) {
    return launch_cluster(selected_simt_kernel<D, kHeads>, dim3(p.splits, p.n_heads / kHeads, p.batch), kSimtThreads, 0, p, s);
}

template <int D>
cudaError_t run_simt_g(const SelectedParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return run_simt<D, 1>(p, s);
        case 2: return run_simt<D, 2>(p, s);
        default: return run_simt<D, 4>(p, s);        // eight heads: two CTAs of four
    }
}

}  // namespace

// As many CTAs as are resident at once (four of four warps per SM), while each
// warp keeps a block.  A step of 16 requests x 4K positions takes 22.2 us so, 29
// with half as many CTAs, 27.3 with twice as many; 64 requests x 2048 positions
// (a CTA per entry and kv head) take 88.8 us so, 89 to 94 with two and four.
int selected_splits(int64_t batch, int n_kv_heads, int64_t top_k, int64_t page_size, int64_t max_len, int sms) {
    const int64_t units = batch * n_kv_heads;
    const int64_t pages = (max_len + page_size - 1) / page_size;
    const int64_t blocks = ((top_k < pages ? top_k : pages) * page_size + kBlk - 1) / kBlk;
    int64_t splits = 4LL * sms / units;
    if (splits > blocks / kMmaWarps) splits = blocks / kMmaWarps;
    if (splits > kMaxSplits) splits = kMaxSplits;
    return splits < 1 ? 1 : static_cast<int>(splits);
}

cudaError_t launch_decode_selected(const SelectedParams &p, int dtype, int head_dim, int group, cudaStream_t s) {
    if (!sparse_supported(dtype, head_dim, group)) return cudaErrorNotSupported;
    if (p.splits < 1 || p.splits > kMaxSplits) return cudaErrorInvalidValue;
    if (dtype == PKV_BF16) return head_dim == 128 ? run_mma_g<128>(p, group, s) : run_mma_g<64>(p, group, s);
    return head_dim == 128 ? run_simt_g<128>(p, group, s) : run_simt_g<64>(p, group, s);
}

}  // namespace pkv
