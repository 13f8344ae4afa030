// pkv_chunk.cu -- attention of each entry's new tokens over its context through
// the page table (pkv_paged_chunk): the fp32 kernel and the join of a context's
// splits.
//
// Row i of entry b, head h sees the positions j <= lim(i) (causal: n - q_len + i,
// else n - 1) and gets
//   o = sum_j softmax_j(scale q . k_j) v_j.
// One pass over the keys with a running maximum m (in base-2 units of the scaled
// score) and sum l; a context that is cut into splits ends in partials o / l and
// (m, l), joined as o = sum_s l_s 2^(m_s - M) o_s / sum_s l_s 2^(m_s - M).
//
// fp32: the tensor cores have no product of 24-bit factors (three bf16 parts of each
// and six products would make one; not built), so this runs on the FMA units.  A CTA
// of 256 threads takes 64 rows (position, head in group; 16 or 32 where an entry has
// no more) and 64 keys at a time; a thread holds a 4 x 4 block of scores and a 4 x
// (D / 16) block of o, so a 16-byte shared-memory load feeds eight FMAs (two lanes
// to an instruction).  K of the next tile is copied while the softmax and P V run, V
// while the next scores do.  4 x 512 tokens at 1K to 2K positions, 32 / 8 heads of
// 128: 1060 us, 40 TFLOP/s of the units' 74 to 80; the loads from shared memory take
// three quarters of the time that the products do.
#include <atomic>
#include <type_traits>

#include "pkv_chunk_join.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

constexpr int kThreads = 256;
constexpr int kTok = 64;

template <int D, int R>
struct Layout {
    static constexpr int kRows = 16 * R;
    // Floats.  Unpadded; a 16-byte chunk c of a row stands at c ^ x, so that the
    // rows that a warp reads at once meet different banks: x is r / R % 2 in Q
    // and P (two row blocks per warp) and r % 8 in K.
    static constexpr int kQ = 0;                      // [kRows][D]
    static constexpr int kK = kQ + kRows * D;         // [kTok][D]
    static constexpr int kV = kK + kTok * D;          // [kTok][D]
    static constexpr int kP = kV + kTok * D;          // [kRows][kTok]
    static constexpr int kFloats = kP + kRows * kTok;
    static constexpr int kBytes = kFloats * 4 + 2 * kTok * 4;   // + slots of two tiles
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 2) chunk_f32_kernel(const __grid_constant__ ChunkParams p) {
    using L = Layout<D, R>;
    constexpr int kRows = L::kRows;
    extern __shared__ __align__(16) float smem[];
    float *sQ = smem + L::kQ, *sK = smem + L::kK, *sV = smem + L::kV, *sP = smem + L::kP;
    int *slots = reinterpret_cast<int *>(smem + L::kFloats);
    constexpr int kChunks = D / 4, kOut = D / 64;       // 16-byte chunks per row; float4 columns of o per thread
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int g = blockIdx.x, split = blockIdx.y % p.n_splits, G = 1 << p.group_shift;
    const ChunkEntry e = entry_of_lane(load_chunk_entry(p, blockIdx.z, g == 0 && blockIdx.y == 0 && tid == 0), 0);
    const int rows = e.q_len << p.group_shift;
    // the entry's last rows, which see most, first
    const int tile = (rows + kRows - 1) / kRows - 1 - static_cast<int>(blockIdx.y / p.n_splits);
    if (tile < 0) return;
    const int row0 = tile * kRows;
    const int last = (min(row0 + kRows, rows) - 1) >> p.group_shift;
    const int kv_lo = split * p.split_len;
    const int kv_end = min(min(kv_lo + p.split_len, e.kv_len), chunk_limit(p, e, last) + 1);
    // nothing to see: zeros, or (cut) nothing that the join would read
    if (kv_end <= kv_lo && p.n_splits > 1) return;
    const int n_tiles = kv_end > kv_lo ? (kv_end - kv_lo + kTok - 1) / kTok : 0;
    const int seen_by_all = chunk_limit(p, e, row0 >> p.group_shift);

    const float *kbase = static_cast<const float *>(p.k_buffer) + (p.layer_row0 * p.n_kv_heads + g) * D;
    const float *vbase = static_cast<const float *>(p.v_buffer) + (p.layer_row0 * p.n_kv_heads + g) * D;
    const int64_t pitch = static_cast<int64_t>(p.n_kv_heads) * D;
    const int32_t *table = p.req_to_page + static_cast<int64_t>(e.req) * p.max_pages;
    auto stage_slots = [&](int t) {                     // of tile t; -1 behind the end
        if (tid >= kTok) return;
        const int j = kv_lo + t * kTok + tid;
        int slot = -1;
        if (j < kv_end) {
            const int i = j / p.page_size, page = __ldg(table + i);
            const bool ok = static_cast<unsigned long long>(static_cast<long long>(page)) < static_cast<unsigned long long>(p.n_pages);
            if (!ok) record_error(p.err, page);
            slot = (ok ? page : 0) * p.page_size + (j - i * p.page_size);
        }
        slots[(t & 1) * kTok + tid] = slot;
    };
    auto copy = [&](float *dst, int mask, const float *base, int t) {
        const int *sl = slots + (t & 1) * kTok;
#pragma unroll
        for (int i = tid; i < kTok * kChunks; i += kThreads) {
            const int r = i / kChunks, c = i % kChunks, slot = sl[r];
            cp_async16(dst + r * D + (c ^ (r & mask)) * 4, slot >= 0 ? base + slot * pitch + c * 4 : base, slot >= 0 ? 16 : 0);
        }
        cp_async_commit();
    };

    if (n_tiles > 0) stage_slots(0);
    for (int i = tid; i < kRows * kChunks; i += kThreads) {
        const int r = i / kChunks, c = i % kChunks, row = row0 + r;
        const float *q = static_cast<const float *>(p.q);
        const bool ok = row < rows;
        const int64_t at = (static_cast<int64_t>(e.qo0 + (row >> p.group_shift)) * p.n_heads + g * G + (row & (G - 1))) * D + c * 4;
        cp_async16(sQ + r * D + (c ^ (r / R & 1)) * 4, ok ? q + at : q, ok ? 16 : 0);
    }
    cp_async_commit();
    __syncthreads();
    if (n_tiles > 0) {
        copy(sK, 7, kbase, 0);
        copy(sV, 0, vbase, 0);
    }

    uint64_t o[R][2 * kOut];                            // two columns each
    float m[R], l[R];
    int lim[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        const int row = row0 + ty * R + r;
        lim[r] = row < rows ? chunk_limit(p, e, row >> p.group_shift) : -1;
#pragma unroll
        for (int c = 0; c < 2 * kOut; ++c) o[r][c] = 0ull;
    }
    for (int t = 0; t < n_tiles; ++t) {
        cp_async_wait<1>();                             // K (and q) have landed, V may be in flight
        if (t + 1 < n_tiles) stage_slots(t + 1);
        __syncthreads();
        // two partial sums per score, of the even and the odd channels
        uint64_t s2[R][4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            ulonglong2 a[R], b[4];
#pragma unroll
            for (int r = 0; r < R; ++r) a[r] = *reinterpret_cast<const ulonglong2 *>(sQ + (ty * R + r) * D + (d ^ (ty & 1) << 2));
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const ulonglong2 *>(sK + (tx + 16 * c) * D + (d ^ (tx & 7) << 2));
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s2[r][c] = f2_fma(a[r].x, b[c].x, s2[r][c]);
                    s2[r][c] = f2_fma(a[r].y, b[c].y, s2[r][c]);
                }
        }
        float s[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float even, odd;
                f2_unpack(s2[r][c], even, odd);
                s[r][c] = even + odd;
            }
        __syncthreads();                                // K's readers are done
        if (t + 1 < n_tiles) copy(sK, 7, kbase, t + 1);
        else cp_async_commit();
        const int j0 = kv_lo + t * kTok;
        const bool masked = j0 + kTok - 1 > min(seen_by_all, kv_end - 1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mt = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[r][c] *= p.scale_log2;
                if (masked && j0 + tx + 16 * c > min(lim[r], kv_end - 1)) s[r][c] = -INFINITY;
                mt = fmaxf(mt, s[r][c]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
            const float mn = fmaxf(m[r], mt);
            const float ref = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: weights 2^-inf = 0
            const float alpha = exp2f(m[r] - ref);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[r][c] = exp2f(s[r][c] - ref);
                sum += s[r][c];
                sP[(ty * R + r) * kTok + ((tx + 16 * c) ^ (ty & 1) << 2)] = s[r][c];
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            m[r] = mn;
            l[r] = l[r] * alpha + sum;
            const uint64_t alpha2 = f2_pack(alpha, alpha);
#pragma unroll
            for (int c = 0; c < 2 * kOut; ++c) o[r][c] = f2_mul(o[r][c], alpha2);
        }
        cp_async_wait<1>();                             // V has landed, the next K may be in flight
        __syncthreads();
        // (two loops: the choices below cost as much as the products)
        auto times_v = [&](auto some) {
            constexpr bool kMasked = decltype(some)::value;
#pragma unroll 2
            for (int k = 0; k < kTok; k += 4) {
                float4 w[R];
#pragma unroll
                for (int r = 0; r < R; ++r) w[r] = *reinterpret_cast<const float4 *>(sP + (ty * R + r) * kTok + (k ^ (ty & 1) << 2));
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int c = 0; c < kOut; ++c) {
                        ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sV + (k + u) * D + tx * 4 + 64 * c);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float x = u == 0 ? w[r].x : u == 1 ? w[r].y : u == 2 ? w[r].z : w[r].w;
                            // a value that the row does not see has no part in its sum, whatever it is
                            const bool seen = !kMasked || j0 + k + u <= lim[r];
                            const uint64_t x2 = f2_pack(x, x);
                            o[r][2 * c] = f2_fma(x2, seen ? v.x : 0ull, o[r][2 * c]);
                            o[r][2 * c + 1] = f2_fma(x2, seen ? v.y : 0ull, o[r][2 * c + 1]);
                        }
                    }
            }
        };
        if (masked) times_v(std::true_type{});
        else times_v(std::false_type{});
        __syncthreads();                                // V's and P's readers are done
        if (t + 1 < n_tiles) copy(sV, 0, vbase, t + 1);
        else cp_async_commit();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int at = row0 + ty * R + r;
        if (at >= rows) continue;
        const int row = e.qo0 + (at >> p.group_shift), head = g * G + (at & (G - 1));
        // a sum of 0 is that of a row that sees nothing here, or -inf alone (the largest
        // weight is 1); the join tells them apart for all pieces together
        const float inv = chunk_inverse(l[r], p.n_splits == 1 && lim[r] >= 0);
        const int64_t unit = chunk_unit(p, split, row, head);
        float *dst = p.n_splits > 1 ? p.o_part + unit * D : static_cast<float *>(p.o) + (static_cast<int64_t>(row) * p.n_heads + head) * D;
#pragma unroll
        for (int c = 0; c < kOut; ++c)
            *reinterpret_cast<float4 *>(dst + tx * 4 + 64 * c) =
                make_float4(f2_lo(o[r][2 * c]) * inv, f2_hi(o[r][2 * c]) * inv, f2_lo(o[r][2 * c + 1]) * inv, f2_hi(o[r][2 * c + 1]) * inv);
        if (p.n_splits > 1 && tx == 0) *reinterpret_cast<float2 *>(p.ml_part + 2 * unit) = make_float2(m[r], l[r]);
    }
}

// The join of the splits: a warp per (row, head).  A split whose first position
// the row does not see has written nothing for it and is not read.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const ChunkEntry e = load_chunk_entry(p, blockIdx.z, false);
    const int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (u >= static_cast<int64_t>(e.q_len) * p.n_heads) return;
    const int i = static_cast<int>(u / p.n_heads), head = static_cast<int>(u - static_cast<int64_t>(i) * p.n_heads);
    const int lim = min(chunk_limit(p, e, i), e.kv_len - 1);
    const int n = lim < 0 ? 0 : lim / p.split_len + 1;
    join_row<T, D>(p, n, [&](int s) { return chunk_unit(p, s, e.qo0 + i, head); }, (static_cast<int64_t>(e.qo0 + i) * p.n_heads + head) * D);
}

template <int D, int R>
cudaError_t run_f32(const ChunkParams &p, int group, cudaStream_t s) {
    using L = Layout<D, R>;
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        e = cudaFuncSetAttribute(chunk_f32_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (e != cudaSuccess) return e;
        attr_done.fetch_or(bit);
    }
    const int tiles = (p.max_q_len * group + L::kRows - 1) / L::kRows;
    chunk_f32_kernel<D, R><<<dim3(p.n_kv_heads, tiles * p.n_splits, p.batch), kThreads, L::kBytes, s>>>(p);
    return cudaGetLastError();
}

// Rows per CTA: 64, or 16 or 32 where an entry has no more.
int f32_rows(int max_q_len, int group) {
    const int64_t rows = static_cast<int64_t>(max_q_len) * group;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

template <int D>
cudaError_t run_f32_rows(const ChunkParams &p, int group, cudaStream_t s) {
    switch (f32_rows(p.max_q_len, group)) {
        case 16: return run_f32<D, 1>(p, group, s);
        case 32: return run_f32<D, 2>(p, group, s);
        default: return run_f32<D, 4>(p, group, s);
    }
}

template <typename T, int D>
cudaError_t run_join(const ChunkParams &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const int64_t units = static_cast<int64_t>(p.max_q_len) * p.n_heads;
    cfg.gridDim = dim3(static_cast<unsigned>((units + kThreads / 32 - 1) / (kThreads / 32)), 1, p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_join_kernel<T, D>, p);
}

}  // namespace

bool chunk_supported(int dtype, int head_dim, int group) {
    return (dtype == PKV_F32 || dtype == PKV_BF16) && (head_dim == 64 || head_dim == 128) &&
           (group == 1 || group == 2 || group == 4 || group == 8);
}

void chunk_plan(ChunkPlan *out, int dtype, int head_dim, int n_kv_heads, int group, int batch, int n_q, int max_q_len, int max_len,
                int sms, size_t room) {
    ChunkPlan &plan = *out;
    plan = ChunkPlan{};
    plan.n_splits = 1;
    plan.split_len = kChunkMaxLen;
    if (dtype == PKV_BF16 && !chunk_wide(max_q_len, group)) {
        // a CTA on every SM, and partials of one row of an item per step along the tiles
        plan.parts = sms > 0 ? sms : 1;
        const size_t units = (static_cast<size_t>(plan.parts) + static_cast<size_t>(batch) * n_kv_heads) * max_q_len * group;
        plan.o_bytes = units * head_dim * sizeof(float);
        plan.ml_bytes = units * 2 * sizeof(float);
        plan.bytes = plan.o_bytes + plan.ml_bytes + static_cast<size_t>(batch) * n_kv_heads * 2 * sizeof(int32_t);
        if (plan.bytes > room) plan.bytes = 0;            // nothing is cut
        return;
    }
    // CTAs per SM, rows and keys per tile of the kernel that the call takes.  On
    // tensor cores a CTA's start and end cost as much as some 800 keys, so the
    // contexts are cut only where one round of CTAs has room for the pieces, of
    // four tiles at least (8 x 64 tokens at 16K positions: 136 us in one round, 150
    // and 152 in up to two and three, 208 uncut; 2 x 192 at 8K 58, 67, 80 and 106;
    // 512 at 64K 391, 408, 376 and 729).  In fp32 a tile takes longer than start
    // and end do: CTAs for twelve rounds, of two tiles at least, which even out
    // entries of different lengths, unless they fill three rounds whole (16 x 1 to
    // 8 tokens at 0.5K to 4K 199 us against 273 for two rounds, 6 x 10 to 200 at up
    // to 2.5K 519 and 650, 13 entries of up to 1777 positions 70.5 and 69.5; 4 x
    // 512 at 2K, three rounds and a half, 1165 in pieces and 1059 whole).
    const bool wide = dtype == PKV_BF16;
    const int64_t per_sm = wide ? 1 : 2, rows = wide ? 256 : f32_rows(max_q_len, group), tok = wide ? 128 : 64;
    const int64_t tiles = (static_cast<int64_t>(max_q_len) * group + rows - 1) / rows;
    const int64_t ctas = tiles * n_kv_heads * batch;
    const int64_t kv_tiles = (static_cast<int64_t>(max_len) + tok - 1) / tok;
    const size_t per_split = static_cast<size_t>(n_q) * n_kv_heads * group;
    const size_t most = per_split > 0 ? room / (per_split * (head_dim + 2) * sizeof(float)) : 0;
    const int64_t round = per_sm * sms;
    int64_t splits = ctas <= 0 ? 1 : wide ? round / ctas : ctas > 3 * round ? 1 : 12 * round / ctas;
    if (splits > kv_tiles / (wide ? 4 : 2)) splits = kv_tiles / (wide ? 4 : 2);
    if (splits > 0 && static_cast<size_t>(splits) > most) splits = static_cast<int64_t>(most);
    if (splits > 65535 / tiles) splits = 65535 / tiles;   // grid y
    if (splits <= 1) return;
    const int64_t per = (kv_tiles + splits - 1) / splits;
    plan.split_len = static_cast<int32_t>(per * tok);
    plan.n_splits = static_cast<int32_t>((kv_tiles + per - 1) / per);
    if (plan.n_splits == 1) return;
    plan.o_bytes = per_split * plan.n_splits * head_dim * sizeof(float);
    plan.ml_bytes = per_split * plan.n_splits * 2 * sizeof(float);
    plan.bytes = plan.o_bytes + plan.ml_bytes;
}

cudaError_t launch_chunk(const ChunkParams &p, int parts, int dtype, int head_dim, int group, cudaStream_t s) {
    if (!chunk_supported(dtype, head_dim, group)) return cudaErrorNotSupported;
    const bool f32 = dtype == PKV_F32;
    if (parts > 0) return launch_chunk_rows(p, parts, head_dim, group, s);
    cudaError_t e = !f32 ? launch_chunk_tc(p, head_dim, group, s) : head_dim == 128 ? run_f32_rows<128>(p, group, s) : run_f32_rows<64>(p, group, s);
    if (e != cudaSuccess || p.n_splits == 1) return e;
    if (f32) return head_dim == 128 ? run_join<float, 128>(p, s) : run_join<float, 64>(p, s);
    return head_dim == 128 ? run_join<__nv_bfloat16, 128>(p, s) : run_join<__nv_bfloat16, 64>(p, s);
}

}  // namespace pkv
