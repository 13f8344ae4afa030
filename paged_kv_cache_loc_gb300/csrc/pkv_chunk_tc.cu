// pkv_chunk_tc.cu -- attention of new tokens through the page table
// (pkv_paged_chunk), bf16, on the 5th-generation tensor cores.
//
// The mathematics is that of pkv_chunk.cu: one pass over the keys with a running
// maximum and sum, O rescaled when the maximum is raised.  This kernel takes
// entries of more than 128 rows (position, head in group); pkv_chunk_rows.cu those
// of fewer.  A CTA takes one kv head of one entry, two tiles of 128 rows, and the
// keys of one split, 128 at a time:
//   S = Q K^T  (tcgen05.mma, fp32 in tensor memory), P = 2^(S - m) as bf16 over
//   S's columns (head_dim 64: beside them), O += P V (P read from tensor memory).
// The two tiles share every K/V tile, and the tensor core works on one while the
// softmax runs on the other.  Every CTA fetches its own K/V tiles: 64 KB in 1.5 us
// on each SM, 6.6 TB/s together, near the 7 to 8 that the SMs fetch at most, from L2
// or not.  4 x 2048 tokens at 8K to 16K, 32 / 8 heads of 128: 914 to 919 us, 1650
// TFLOP/s; of 64: 790 us, 957 TFLOP/s.
// Warps hand over through mbarriers, every wait bounded:
//   8 softmax warps, one thread per row: the row maximum needs no exchange;
//   one warp that issues the products;
//   one warp that copies K and V with TMA.  Positions of a page are consecutive
//     rows of the pool, so a box of as many rows as the largest power of two in
//     page_size never crosses a page; pages of other sizes are gathered four
//     rows at a time (tile::gather4).  All rows that a copy names lie in the
//     pool: behind the split's end it reads page 0, whose rows then count for
//     nothing;
//   two warps that look at the V tiles which some row of the CTA does not see
//     wholly: a product with the weight 0 must not meet a value that is not
//     finite.  Rows behind the end become 0; a value that is not finite is
//     taken out and noted, and the epilogue adds it to the rows that see it.
#include <atomic>

#include "pkv_chunk_tc.cuh"

namespace pkv {
namespace {

constexpr int kRows = 128;                  // query rows per tile (tensor-memory lanes)
constexpr int kPair = 2 * kRows;            // query rows per CTA
constexpr int kGuarded = 3;                 // V tiles that are looked at, at most (256 positions)

template <int D>
struct Tc {
    static constexpr int kTok = 128, kThreads = 384;
    static constexpr int kSlots = D == 64 ? 4 : 2;      // K tiles and V tiles in shared memory
    static constexpr bool kOwnP = D == 64;              // P has columns of its own
    static constexpr int kMmaWarp = 0, kCopyWarp = 1, kGuardWarp = 2, kSoftmaxWarp = 4;
    static constexpr int kQBytes = kRows * D * 2, kTileBytes = kTok * D * 2;
    static constexpr int kSmemQ = 0, kSmemK = 2 * kQBytes, kSmemV = kSmemK + kSlots * kTileBytes;
    static constexpr int kSmemBar = kSmemV + kSlots * kTileBytes;
    // barriers
    static constexpr int kKFull = 0, kKEmpty = kSlots, kVFull = 2 * kSlots, kVEmpty = 3 * kSlots;
    static constexpr int kVRaw = 4 * kSlots, kVClean = 5 * kSlots;      // in VFull's place for tiles that are looked at
    static constexpr int kSFull = 6 * kSlots, kPFull = kSFull + 2, kODone = kPFull + 2, kSRead = kODone + 2;
    static constexpr int kQFull = kSRead + 2, kBars = kQFull + 1;
    static constexpr int kSmemTmem = kSmemBar + kBars * 8, kSmemAbort = kSmemTmem + 4, kSmemBad = kSmemAbort + 4;
    static constexpr int kBadWords = kGuarded * kTok / 32 + 1;      // bits of rows, then: any
    static constexpr int kBytes = kSmemBad + kBadWords * 4 + 1024;  // + alignment slack
    // registers: the launch's, and how the warps share them
    // (a softmax thread holds 128 scores)
    static constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
    static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "no more than the launch holds");
    // tensor memory
    static constexpr uint32_t kCols = 512;
    __device__ static constexpr uint32_t s_col(int X) { return X * 256; }
    __device__ static constexpr uint32_t o_col(int X) { return X * 256 + 128; }
    __device__ static constexpr uint32_t p_col(int X) { return kOwnP ? X * 256 + 192 : s_col(X); }
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(384, 1)
chunk_tc_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ Maps maps, const int box) {
    using bf16 = __nv_bfloat16;
    using L = Tc<D>;
    constexpr int kTok = L::kTok, kChunks = D / 8, kSlots = L::kSlots;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t s_base = smem_u32(sm);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + L::kSmemAbort);
    uint32_t *s_bad = reinterpret_cast<uint32_t *>(sm + L::kSmemBad);
    auto bar = [&](int i) -> uint32_t { return s_base + L::kSmemBar + 8 * i; };

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int g = blockIdx.x, shift = p.group_shift, G = 1 << shift, split = blockIdx.y % p.n_splits;
    const ChunkEntry e = load_longest_entry(p, blockIdx.z, g == 0 && blockIdx.y == 0 && warp == 0);
    const int rows = e.q_len << shift;
    // the entry's last rows, which see most, first
    const int tile = (rows + kPair - 1) / kPair - 1 - static_cast<int>(blockIdx.y / p.n_splits);
    if (tile < 0) return;
    const int row0 = tile * kPair;
    const int kv_lo = split * p.split_len;
    // keys [kv_lo, end) that the rows up to `row` see in this split
    auto end_of = [&](int row) -> int { return min(min(kv_lo + p.split_len, e.kv_len), chunk_limit(p, e, row >> shift) + 1); };
    int n_x[2];                                         // tiles of keys of each query tile
#pragma unroll
    for (int X = 0; X < 2; ++X) {
        const int r0 = row0 + X * kRows, end = r0 < rows ? end_of(min(r0 + kRows, rows) - 1) : kv_lo;
        n_x[X] = end > kv_lo ? (end - kv_lo + kTok - 1) / kTok : 0;
    }
    const int kv_end = max(kv_lo, end_of(min(row0 + kPair, rows) - 1));
    const int n_tiles = (kv_end - kv_lo + kTok - 1) / kTok;
    if (n_tiles == 0 && p.n_splits > 1) return;       // nothing to see: the join does not read this split
    // from tile `guard` on, some row does not see all of a tile
    const int all_see = min(chunk_limit(p, e, row0 >> shift), kv_end - 1);
    const int guard = all_see < kv_lo ? 0 : (all_see + 1 - kv_lo) / kTok;

    auto slot_of = [&](int j) -> int {
        const int i = j / p.page_size, page = __ldg(p.req_to_page + static_cast<int64_t>(e.req) * p.max_pages + i);
        const bool ok = static_cast<unsigned long long>(static_cast<long long>(page)) < static_cast<unsigned long long>(p.n_pages);
        if (!ok) record_error(p.err, page);
        return (ok ? page : 0) * p.page_size + (j - i * p.page_size);
    };
    // ---- copies: a lane takes a box of rows, or four rows.  The first rows are
    // looked up before the barriers are made.
    const int per = box > 0 ? box : 4;
    const bool active = lane < kTok / per;
    int next[4] = {0, 0, 0, 0};
    auto fetch = [&](int t) {
        if (!active || t >= n_tiles) return;
        const int j = kv_lo + t * kTok + lane * per;
        if (box > 0) {
            next[0] = j < kv_end ? slot_of(j) : 0;
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) next[u] = j + u < kv_end ? slot_of(j + u) : 0;
        }
    };
    if (warp == L::kCopyWarp) fetch(0);

    // ---- barriers, tensor memory
    if (tid == 0) {
        for (int i = 0; i < L::kBars; ++i) {
            uint32_t count = 1;
            if (i >= L::kVClean && i < L::kSFull) count = 2;
            else if ((i >= L::kPFull && i < L::kODone) || (i >= L::kSRead && i < L::kQFull)) {    // the tile's warps that hold rows
                const int left = rows - row0 - ((i - L::kPFull) & 1) * kRows;
                count = max(1, (min(left, kRows) + 31) / 32);
            } else if (i == L::kQFull) count = 256;
            mbar_init(bar(i), count);
        }
        for (int i = 0; i < L::kBadWords; ++i) s_bad[i] = 0;
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == L::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(s_base + L::kSmemTmem), "r"(L::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(sm + L::kSmemTmem), 0);
    auto give_up = [&](int code) {
        if (lane == 0 && *s_abort == 0) {
            *s_abort = 1;
            record_error(p.err, code);
        }
    };
    // phase of slot barriers at tile t
    auto phase = [](int t) -> uint32_t { return (t / kSlots) & 1; };
    // The copies of V tile t complete a barrier of their own from tile `guard` on:
    // each barrier's phases are waited for one after the other.
    auto v_landed = [&](int t) -> uint32_t { return bar((t < guard ? L::kVFull : L::kVRaw) + t % kSlots); };
    auto v_phase = [&](int t) -> uint32_t { return t < guard ? phase(t) : phase(t - guard); };

    if (warp < L::kSoftmaxWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(L::kOtherRegs));
        if (warp == L::kCopyWarp) {
            // ================= copies
            auto issue = [&](const CUtensorMap *map, uint32_t dst, uint32_t full, const int (&row)[4]) {
                if (lane == 0) expect_bytes(full, L::kTileBytes);
                __syncwarp();
                if (!active) return;
                if (box > 0) {
                    copy_box(dst + lane * per * (D * 2), map, g * (D / 64), row[0] >> 3, full);
                } else {
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        copy_rows4(dst + (lane >> 1) * (D * 16) + h * 1024 + (lane & 1) * 512, map, g * D + h * 64, row, full);
                }
            };
            int issued_k = 0, issued_v = 0;
            for (int t = 0; t < n_tiles; ++t) {
                const int row[4] = {next[0], next[1], next[2], next[3]};
                fetch(t + 1);
                const int slot = t % kSlots;
                bool ok = *s_abort == 0 && bar_wait(bar(L::kKEmpty + slot), phase(t) ^ 1);
                if (!__all_sync(0xffffffffu, ok)) { give_up(-5001); break; }
                issue(&maps.k, s_base + L::kSmemK + slot * L::kTileBytes, bar(L::kKFull + slot), row);
                issued_k = t + 1;
                ok = *s_abort == 0 && bar_wait(bar(L::kVEmpty + slot), phase(t) ^ 1);
                if (!__all_sync(0xffffffffu, ok)) { give_up(-5002); break; }
                issue(&maps.v, s_base + L::kSmemV + slot * L::kTileBytes, v_landed(t), row);
                issued_v = t + 1;
            }
            // no copy is in flight when the CTA ends, also after a wait that gave up
            for (int t = max(0, issued_k - kSlots); t < issued_k; ++t) bar_wait(bar(L::kKFull + t % kSlots), phase(t));
            for (int t = max(0, issued_v - kSlots); t < issued_v; ++t) bar_wait(v_landed(t), v_phase(t));
            // and no release
            bool reached = issued_v == n_tiles;
            for (int t = max(0, n_tiles - kSlots); reached && t < n_tiles; ++t)
                reached = *s_abort == 0 && bar_wait(bar(L::kKEmpty + t % kSlots), phase(t)) && bar_wait(bar(L::kVEmpty + t % kSlots), phase(t));
            __syncwarp();
        } else if (warp == L::kMmaWarp) {
            // ================= products: one thread issues them all.  It blocks
            // while the tensor core is busy, so what it does in between is
            // time in which the tensor core runs dry: it waits for K and V
            // while the products before them run, and looks at nothing else.
            if (n_tiles > 0) {
                const uint32_t id_s = idesc(kRows, kTok, 0), id_o = idesc(kRows, D, 1);
                const uint64_t dq = sdesc(s_base + L::kSmemQ, 16, D * 16), dk = sdesc(s_base + L::kSmemK, 16, D * 16);
                const uint64_t dv = sdesc(s_base + L::kSmemV, 1024, D * 16);
                const uint32_t hi = static_cast<uint32_t>(dq >> 32), v_hi = static_cast<uint32_t>(dv >> 32);
                const uint32_t q_lo = static_cast<uint32_t>(dq), k_lo = static_cast<uint32_t>(dk), v_lo = static_cast<uint32_t>(dv);
                auto issue_s = [&](int X, int slot) {
                    if (!elect()) return;
                    const uint32_t qa = q_lo + X * (L::kQBytes >> 4), ka = k_lo + slot * (L::kTileBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_f16(tmem + L::s_col(X), desc_at(qa + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), hi),
                                desc_at(ka + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), hi), id_s, ks > 0);
                    mma_commit(bar(L::kSFull + X));
                };
                auto issue_pv = [&](int X, int slot, bool acc) {
                    if (!elect()) return;
                    const uint32_t va = v_lo + slot * (L::kTileBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < kTok / 16; ++ks)
                        mma_f16_ta(tmem + L::o_col(X), tmem + L::p_col(X) + ks * 8, desc_at(va + ks * (2 * D * 16 >> 4), v_hi), id_o,
                                   (acc || ks > 0) ? 1u : 0u);
                };
                auto commit = [&](int i) {
                    if (elect()) mma_commit(bar(i));
                };
                auto wait_k = [&](int t) -> bool { return wait_fast(bar(L::kKFull + t % kSlots), phase(t)); };
                auto wait_v = [&](int t) -> bool { return wait_fast(bar((t < guard ? L::kVFull : L::kVClean) + t % kSlots), v_phase(t)); };
                bool ok = wait_fast(bar(L::kQFull), 0) && wait_k(0);
                if (ok) {
                    fence_after();
                    if (n_x[0] > 0) issue_s(0, 0);
                    if (n_x[1] > 0) issue_s(1, 0);
                    commit(L::kKEmpty);
                    ok = L::kOwnP || (wait_v(0) && (n_tiles == 1 || wait_k(1)));
                }
                // P in columns of its own (head_dim 64 leaves 64): S of the next tiles runs
                // as soon as the last is read, while the softmax works on it (16 chunks of
                // up to 448 tokens over up to 1500 states 37.9 us, 40.5 with P over S; 8 x
                // 512 tokens at 2K 96.0 and 96.7, but 4 x 2048 at 8K to 16K 792 and 781)
                for (int j = 0; L::kOwnP && ok && j < n_tiles; ++j) {
                    const int slot = j % kSlots, slot1 = (j + 1) % kSlots;
                    if (j + 1 < n_tiles) {
                        if (!wait_k(j + 1)) { ok = false; break; }
#pragma unroll
                        for (int X = 0; X < 2; ++X)
                            if (ok && j + 1 < n_x[X]) {
                                ok = wait_fast(bar(L::kSRead + X), j & 1);
                                fence_after();
                                if (ok) issue_s(X, slot1);
                            }
                        if (!ok) break;
                        commit(L::kKEmpty + slot1);
                    }
                    if (!wait_v(j)) { ok = false; break; }
#pragma unroll
                    for (int X = 0; X < 2; ++X)
                        if (ok && j < n_x[X]) {
                            ok = wait_fast(bar(L::kPFull + X), j & 1);
                            fence_after();
                            if (!ok) continue;
                            issue_pv(X, slot, j > 0);
                            commit(L::kODone + X);
                        }
                    commit(L::kVEmpty + slot);
                }
                for (int j = 0; !L::kOwnP && ok && j < n_tiles; ++j) {
                    const int slot = j % kSlots, slot1 = (j + 1) % kSlots;
                    const bool more = j + 1 < n_tiles;
                    if (j < n_x[0]) {
                        if (!wait_fast(bar(L::kPFull), j & 1)) { ok = false; break; }
                        fence_after();
                        issue_pv(0, slot, j > 0);
                        if (j == n_x[0] - 1) commit(L::kODone);
                    }
                    if (j + 1 < n_x[0]) issue_s(0, slot1);
                    if (more && !wait_v(j + 1)) { ok = false; break; }
                    if (j < n_x[1]) {
                        if (!wait_fast(bar(L::kPFull + 1), j & 1)) { ok = false; break; }
                        fence_after();
                        issue_pv(1, slot, j > 0);
                        if (j == n_x[1] - 1) commit(L::kODone + 1);
                    }
                    commit(L::kVEmpty + slot);
                    if (j + 1 < n_x[1]) issue_s(1, slot1);
                    if (more) commit(L::kKEmpty + slot1);
                    if (j + 2 < n_tiles) ok = wait_k(j + 2);
                }
                if (!ok) give_up(-5003);
            }
            __syncwarp();
        } else {
            // ================= V tiles that not every row sees wholly
            for (int t = guard; t < n_tiles; ++t) {
                const bool ok = *s_abort == 0 && bar_wait(v_landed(t), v_phase(t));
                if (!__all_sync(0xffffffffu, ok)) { give_up(-5008); break; }
                unsigned char *v = sm + L::kSmemV + (t % kSlots) * L::kTileBytes;
                for (int r = tid - L::kGuardWarp * 32; r < kTok; r += 64) {
                    const int j = kv_lo + t * kTok + r;
                    if (j <= all_see) continue;
                    if (j >= kv_end) {
                        for (int c = 0; c < kChunks; ++c) *reinterpret_cast<uint4 *>(v + sw_at<D>(r, c)) = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    bool bad = false;
#pragma unroll 4
                    for (int c = 0; c < kChunks; ++c) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(v + sw_at<D>(r, c));
                        bad |= not_finite(w.x) || not_finite(w.y) || not_finite(w.z) || not_finite(w.w);
                    }
                    if (bad) {
                        for (int i = 0; i < D; ++i) {
                            uint16_t *x = reinterpret_cast<uint16_t *>(v + sw_at<D>(r, i / 8)) + (i & 7);
                            if ((*x & 0x7f80u) == 0x7f80u) *x = 0;
                        }
                        atomicOr(s_bad + ((t - guard) * kTok + r) / 32, 1u << (r & 31));
                        s_bad[L::kBadWords - 1] = 1;
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kVClean + t % kSlots));
            }
        }
    } else {
        // ================= softmax: the rows of tile X, a thread each
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(L::kSoftmaxRegs));
        const int X = (warp - L::kSoftmaxWarp) >> 2, row = tid & (kRows - 1), R0 = row0 + X * kRows, R = R0 + row;
        {
            // The maximum is of the products, so a scale below 0 is taken into q,
            // and one of 0 makes q 0.
            const uint32_t q_and = p.scale_log2 == 0.f ? 0u : ~0u, q_xor = p.scale_log2 < 0.f ? 0x80008000u : 0u;
            const bf16 *q = static_cast<const bf16 *>(p.q);
            // (all of a thread's chunks on their way before the first is stored: one
            // round trip in front of the first product)
            uint4 w[kChunks];
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                const int i = row + k * kRows, r = i / kChunks, ch = i % kChunks, Rq = R0 + r;
                w[k] = make_uint4(0u, 0u, 0u, 0u);
                if (Rq < rows)
                    w[k] = *reinterpret_cast<const uint4 *>(
                        q + (static_cast<int64_t>(e.qo0 + (Rq >> shift)) * p.n_heads + g * G + (Rq & (G - 1))) * D + ch * 8);
            }
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                const int i = row + k * kRows, r = i / kChunks, ch = i % kChunks;
                w[k].x = (w[k].x & q_and) ^ q_xor, w[k].y = (w[k].y & q_and) ^ q_xor;
                w[k].z = (w[k].z & q_and) ^ q_xor, w[k].w = (w[k].w & q_and) ^ q_xor;
                *reinterpret_cast<uint4 *>(sm + L::kSmemQ + X * L::kQBytes + sw_at<D>(r, ch)) = w[k];
            }
            fence_async_smem();
            mbar_arrive(bar(L::kQFull));
        }
        const int mine = X ? n_x[1] : n_x[0];   // tiles
        const bool busy = R0 + (warp & 3) * 32 < rows;                     // the warp holds rows
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + L::o_col(X) + lane_off;
        const int lim = R < rows ? min(chunk_limit(p, e, R >> shift), e.kv_len - 1) : -1;
        const float sc = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
        float m = -INFINITY, l = 0.f;
        bool live = busy;
        // A look at a barrier ahead of its wait, whose answer takes some 200 cycles while
        // the tensor core reads shared memory (head_dim 64, 4 x 2048 tokens at 8K to
        // 16K: 792 us, 795 without; 16 chunks of up to 448 tokens 37.9 and 38.8).
        auto look = [&](int i, int parity) -> bool {
            uint32_t ok;
            asm volatile(
                "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                " selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(ok)
                : "r"(bar(i)), "r"(parity)
                : "memory");
            return ok != 0;
        };
        for (int j = 0; live && j < mine; ++j) {
            bool ok = *s_abort == 0 && bar_wait(bar(L::kSFull + X), j & 1);
            if (!__all_sync(0xffffffffu, ok)) { give_up(-5009); live = false; break; }
            fence_after();
            const uint32_t t_s = tmem + L::s_col(X) + lane_off;
            float sv[kTok / 64][64];
#pragma unroll
            for (int h = 0; h < kTok / 64; ++h) tmem_ld64(t_s + h * 64, sv[h]);
            if (L::kOwnP) {                            // the next S may come
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kSRead + X));
            }
            auto s = [&](int i) -> float & { return sv[i >> 6][i & 63]; };
            const int j0 = kv_lo + j * kTok;
            if (j0 + kTok - 1 > lim) {
#pragma unroll
                for (int i = 0; i < kTok; ++i)
                    if (j0 + i > lim) s(i) = -INFINITY;
            }
            const bool pv_done = L::kOwnP && j > 0 && look(L::kODone + X, (j - 1) & 1);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kTok; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s(i), s(i + 1));
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
            // The reference is raised only when the tile's maximum exceeds it by
            // 2^8, so weights stay below 2^8 and O is rescaled rarely.
            const bool raise = mt > m + kRescale || (m == -INFINITY && mt != -INFINITY);
            const bool touch = raise && j > 0 && m != -INFINITY;
            const float alpha = raise ? exp2f(m - mt) : 1.f;
            if (L::kOwnP && j > 0) {                   // P V of the tile before: O and P's place
                if (!__all_sync(0xffffffffu, pv_done)) {
                    ok = *s_abort == 0 && bar_wait(bar(L::kODone + X), (j - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) { give_up(-5010); live = false; break; }
                }
                fence_after();
            }
            if (__any_sync(0xffffffffu, touch)) {      // (else P V of the tile before came before this S)
                const float f = touch ? alpha : 1.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    tmem_ld32(t_o + c, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= f;
                    tmem_st32(t_o + c, v);
                }
            }
            if (raise) {
                l *= alpha;
                m = mt;
            }
            const float neg = m == -INFINITY ? -INFINITY : -m;      // nothing seen yet: weights 0
            const uint64_t sc2 = f2_pack(sc, sc), neg2 = f2_pack(neg, neg);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < kTok; c += 16) {
                uint32_t pk[8];
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(s(c + i), s(c + i + 1)), sc2, neg2), x0, x1);
                    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                    sum[(i >> 1) & 1] = f2_add(sum[(i >> 1) & 1], f2_pack(p0, p1));
                    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                    pk[i >> 1] = *reinterpret_cast<const uint32_t *>(&h);
                }
                tmem_st8u(tmem + L::p_col(X) + lane_off + c / 2, pk);
            }
            float a0, a1, a2, a3;
            f2_unpack(sum[0], a0, a1);
            f2_unpack(sum[1], a2, a3);
            l += (a0 + a1) + (a2 + a3);
            asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kPFull + X));
        }
        // ---- epilogue: O is final once its last product is done
        if (busy && live) {     // (nothing to see: the query tile, whose place the rows go through)
            const bool ok = *s_abort == 0 && bar_wait(bar(mine > 0 ? L::kODone + X : L::kQFull), L::kOwnP && mine > 0 ? (mine - 1) & 1 : 0);
            if (!__all_sync(0xffffffffu, ok)) give_up(-5011), live = false;
        }
        fence_after();
        if (__all_sync(0xffffffffu, busy && live && *s_abort == 0 && (mine > 0 || p.n_splits == 1))) {
            const float inv = chunk_inverse(l, p.n_splits == 1 && lim >= 0);
            const bool some_bad = mine > 0 && *static_cast<volatile uint32_t *>(s_bad + L::kBadWords - 1) != 0;
            // columns [c0, c0 + 32) of this row
            auto load_o = [&](int c0, float (&v)[32]) {
                __syncwarp();
                if (mine == 0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                    return;
                }
                tmem_ld32(t_o + c0, v);
                if (some_bad) {     // values that are not finite, for the rows that see them
                    for (int w = 0; w < kGuarded * kTok / 32; ++w)
                        for (uint32_t bits = s_bad[w]; bits; bits &= bits - 1) {
                            const int j = kv_lo + guard * kTok + w * 32 + __ffs(bits) - 1;
                            if (j > lim) continue;
                            const bf16 *x = static_cast<const bf16 *>(p.v_buffer) +
                                            ((p.layer_row0 + slot_of(j)) * p.n_kv_heads + g) * D + c0;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float f = __bfloat162float(x[i]);
                                if (!isfinite(f)) v[i] += f;
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= inv;
            };
            // The warp's rows go through shared memory (its part of the query
            // tile, whose last product is done), 16-byte chunk c of row r at
            // c ^ (r % 8), so that whole row pieces are stored.
            unsigned char *stg = sm + L::kSmemQ + X * L::kQBytes + (warp & 3) * 32 * D * 2;
            const int R_warp = R0 + (warp & 3) * 32;
            if (p.n_splits == 1) {
                constexpr int kCh = D / 8;
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float v[32];
                    load_o(c0, v);
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(v[q4 * 8 + 2 * i], v[q4 * 8 + 2 * i + 1]);
                            w[i] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        *reinterpret_cast<uint4 *>(stg + lane * D * 2 + (((c0 / 8 + q4) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kCh; ++i) {
                    const int r = i * (32 / kCh) + lane / kCh, c = lane % kCh, Rr = R_warp + r;
                    if (Rr < rows)
                        *reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.o) +
                                                   (static_cast<int64_t>(e.qo0 + (Rr >> shift)) * p.n_heads + g * G + (Rr & (G - 1))) * D + c * 8) =
                            *reinterpret_cast<const uint4 *>(stg + r * D * 2 + ((c ^ (r & 7)) << 4));
                }
            } else {
                constexpr int kCh = D / 8;          // chunks of half a row of fp32
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int c0 = 0; c0 < D / 2; c0 += 32) {
                        float v[32];
                        load_o(half * (D / 2) + c0, v);
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4)
                            *reinterpret_cast<float4 *>(stg + lane * D * 2 + (((c0 / 4 + q4) ^ (lane & 7)) << 4)) =
                                make_float4(v[q4 * 4], v[q4 * 4 + 1], v[q4 * 4 + 2], v[q4 * 4 + 3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kCh; ++i) {
                        const int r = i * (32 / kCh) + lane / kCh, c = lane % kCh, Rr = R_warp + r;
                        if (Rr < rows)
                            *reinterpret_cast<float4 *>(p.o_part + chunk_unit(p, split, e.qo0 + (Rr >> shift), g * G + (Rr & (G - 1))) * D +
                                                        half * (D / 2) + c * 4) =
                                *reinterpret_cast<const float4 *>(stg + r * D * 2 + ((c ^ (r & 7)) << 4));
                    }
                    __syncwarp();
                }
                if (R < rows)
                    *reinterpret_cast<float2 *>(p.ml_part + 2 * chunk_unit(p, split, e.qo0 + (R >> shift), g * G + (R & (G - 1)))) =
                        make_float2(m, l);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == L::kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(L::kCols));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

template <int D>
cudaError_t run(const ChunkParams &p, int group, cudaStream_t s) {
    using L = Tc<D>;
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        e = cudaFuncSetAttribute(chunk_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (e != cudaSuccess) return e;
        // the warps' shares add up to the launch's registers: fewer, and they would wait for more
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, chunk_tc_kernel<D>);
        if (e != cudaSuccess) return e;
        if (attr.numRegs < L::kLaunchRegs) return cudaErrorNotSupported;
        attr_done.fetch_or(bit);
    }
    const int box = box_rows(p.page_size, L::kTok);
    Maps maps;
    if (!pool_maps(&maps, p, D, box)) return cudaErrorInvalidValue;
    const int tiles = (p.max_q_len * group + kPair - 1) / kPair;
    chunk_tc_kernel<D><<<dim3(p.n_kv_heads, tiles * p.n_splits, p.batch), L::kThreads, L::kBytes, s>>>(p, maps, box);
    return cudaGetLastError();
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled f = known.load();
    if (!f) {
        void *entry = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &entry, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeTiled>(entry);
        known.store(f);
    }
    return f;
}

// One layer of the pool.  Boxes: 64 columns x 8 rows x the halves of a head x
// groups of 8 rows, in the tile's order; single rows: a matrix of `size` rows.
bool pool_map(CUtensorMap *map, const void *base, const ChunkParams &p, int D, int box) {
    const EncodeTiled f = encoder();
    if (!f) return false;
    const cuuint64_t width = static_cast<cuuint64_t>(p.n_kv_heads) * D, row = width * 2, size = static_cast<cuuint64_t>(p.size);
    const cuuint64_t dims4[4] = {64, 8, width / 64, size / 8}, dims2[2] = {width, size};
    const cuuint64_t strides4[3] = {row, 128, 8 * row}, strides2[1] = {row};
    const cuuint32_t box4[4] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(box / 8)}, box2[2] = {64, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    void *at = const_cast<char *>(static_cast<const char *>(base) + static_cast<size_t>(p.layer_row0) * row);
    return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, box > 0 ? 4 : 2, at, box > 0 ? dims4 : dims2, box > 0 ? strides4 : strides2,
             box > 0 ? box4 : box2, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool pool_maps(Maps *maps, const ChunkParams &p, int D, int box) {
    return pool_map(&maps->k, p.k_buffer, p, D, box) && pool_map(&maps->v, p.v_buffer, p, D, box);
}

bool chunk_wide(int max_q_len, int group) { return static_cast<int64_t>(max_q_len) * group > kRows; }

cudaError_t launch_chunk_tc(const ChunkParams &p, int head_dim, int group, cudaStream_t s) {
    return head_dim == 128 ? run<128>(p, group, s) : run<64>(p, group, s);
}

}  // namespace pkv
