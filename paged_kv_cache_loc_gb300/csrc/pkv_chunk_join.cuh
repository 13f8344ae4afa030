// pkv_chunk_join.cuh -- how the chunk attention joins the pieces of a context, and
// how the kernel for few rows deals out its tiles (internal).
#pragma once

#include "pkv_chunk.cuh"

namespace pkv {

// W key tiles over at most `most` CTAs, two each at least where there are so
// many: CTA c takes [begin(c), begin(c + 1)).
struct ChunkDeal {
    long long tiles;
    int most;
    __device__ __forceinline__ int parts() const {
        const long long x = (tiles + 1) / 2;
        return x < most ? (x < 1 ? 1 : static_cast<int>(x)) : most;
    }
    __device__ __forceinline__ long long begin(int c) const { return tiles * c / parts(); }
};

// Pieces of an item whose first and last tile the CTAs `first` and `last` of `parts`
// list; 0 where one CTA has it whole.  A CTA whose wait gave up has not listed the
// rest of its items: what stands in the workspace for them may be anything, and a
// pair that no CTAs can have is passed over (the call ends with its error code).
__host__ __device__ inline int item_pieces(int first, int last, int parts) {
    return first >= 0 && first < last && last < parts ? last - first + 1 : 0;
}

// o[at ..] = sum_s l_s 2^(m_s - M) o_s / sum_s l_s 2^(m_s - M) over the n pieces of a
// row, piece s at unit(s), by a warp; n = 0 for a row that sees nothing.
template <typename T, int D, typename Unit>
__device__ __forceinline__ void join_row(const ChunkParams &p, int n, Unit unit, int64_t at) {
    constexpr int kPer = D / 32, kLoads = 16;           // elements per lane, pieces in flight
    const int lane = threadIdx.x & 31;
    float top = -INFINITY, sum = 0.f, acc[kPer] = {};
    float v[kLoads][kPer];
    auto load = [&](int s0) {
#pragma unroll
        for (int s = 0; s < kLoads; ++s) {
            if (s0 + s >= n) break;
            const float *src = p.o_part + unit(s0 + s) * D + lane * kPer;
            if constexpr (kPer == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
                v[s][0] = x.x, v[s][1] = x.y, v[s][2] = x.z, v[s][3] = x.w;
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
                v[s][0] = x.x, v[s][1] = x.y;
            }
        }
    };
    for (int s0 = 0; s0 < n; s0 += 32) {                // the pieces' (m, l), a lane each
        load(s0);                                       // (the first of the pieces beside them)
        float m = -INFINITY, l = 0.f;
        if (s0 + lane < n) {
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.ml_part + 2 * unit(s0 + lane)));
            m = ml.x;
            l = ml.y;
        }
        float mt = m;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
        const float mn = fmaxf(top, mt), ref = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(top - ref);
        const float w = l * exp2f(m - ref);
        top = mn;
        float ws = w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
        sum = sum * alpha + ws;
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] *= alpha;
#pragma unroll
        for (int h = 0; h < 32 / kLoads; ++h) {
            if (h > 0 && s0 + h * kLoads < n) load(s0 + h * kLoads);
#pragma unroll
            for (int s = 0; s < kLoads; ++s) {
                const float f = __shfl_sync(0xffffffffu, w, h * kLoads + s);
                if (s0 + h * kLoads + s >= n) continue;
#pragma unroll
                for (int c = 0; c < kPer; ++c) acc[c] = fmaf(f, v[s][c], acc[c]);
            }
        }
    }
    const float inv = chunk_inverse(sum, n > 0);
    T *dst = static_cast<T *>(p.o) + at + lane * kPer;
#pragma unroll
    for (int c = 0; c < kPer; ++c) dst[c] = Elem<T>::from_f(acc[c] * inv);
}

}  // namespace pkv
