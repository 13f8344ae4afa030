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
    // the largest c with begin(c) <= x
    __device__ __forceinline__ int owner(long long x) const { return static_cast<int>(((x + 1) * parts() - 1) / tiles); }
};

// o[at ..] = sum_s l_s 2^(m_s - M) o_s / sum_s l_s 2^(m_s - M) over the n pieces of a
// row, piece s at unit(s), by a warp.
template <typename T, int D, typename Unit>
__device__ __forceinline__ void join_row(const ChunkParams &p, int n, Unit unit, int64_t at) {
    constexpr int kPer = D / 32;                        // elements per lane
    const int lane = threadIdx.x & 31;
    float top = -INFINITY, sum = 0.f, acc[kPer] = {};
    for (int s0 = 0; s0 < n; s0 += 32) {                // the pieces' (m, l), a lane each
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
        const int cnt = min(32, n - s0);
#pragma unroll 8
        for (int s = 0; s < cnt; ++s) {
            const float f = __shfl_sync(0xffffffffu, w, s);
            const float *src = p.o_part + unit(s0 + s) * D + lane * kPer;
            if constexpr (kPer == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                acc[0] = fmaf(f, v.x, acc[0]);
                acc[1] = fmaf(f, v.y, acc[1]);
                acc[2] = fmaf(f, v.z, acc[2]);
                acc[3] = fmaf(f, v.w, acc[3]);
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                acc[0] = fmaf(f, v.x, acc[0]);
                acc[1] = fmaf(f, v.y, acc[1]);
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    T *dst = static_cast<T *>(p.o) + at + lane * kPer;
#pragma unroll
    for (int c = 0; c < kPer; ++c) dst[c] = Elem<T>::from_f(acc[c] * inv);
}

}  // namespace pkv
