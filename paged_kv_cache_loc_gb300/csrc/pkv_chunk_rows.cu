// pkv_chunk_rows.cu -- attention of few new tokens (up to 128 rows of position and
// head in group per entry: drafts to verify, single tokens) through the page
// table (pkv_paged_chunk), bf16, on the 5th-generation tensor cores.
//
// Mathematics, tiles, copies and the care for values that are not finite are
// those of pkv_chunk_tc.cu, with one tile of 128 query rows (mostly empty: the
// tensor core is not what bounds) and key tiles of 128.  Here the memory's rate
// bounds, so nothing may interrupt the stream of K and V:
//   - one CTA per SM, and the key tiles of all items (entry, kv head), one after
//     the other, are dealt out to them evenly: CTA c takes tiles [W c / P, W (c +
//     1) / P) of the W, a run of segments, each a piece of one item;
//   - the copies run on over the segments' borders, 192 KB ahead, while the query
//     tile changes; O has two places, so that a segment's products follow those
//     of the segment before while that one's O is written.
// An item that lies in one CTA is written to o; the pieces of the others go to
// the workspace, piece of item i in CTA c at c + i (each step along the tiles
// raises one of the two), and are joined.  Without room in the workspace a CTA
// takes the items that begin among its tiles, whole.
//
// Warps: products, copies (and the list of segments), query tiles, V tiles that
// not every row sees, four for softmax and output.  The list goes through a ring
// in shared memory.
#include <atomic>

#include "pkv_chunk_join.cuh"
#include "pkv_chunk_tc.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 128;
constexpr int kRows = 128;
constexpr int kSegs = 8;                    // places of the segments' ring
constexpr int kAhead = 3;                   // segments listed before their copies begin
constexpr int kGuarded = 3;                 // V tiles of a segment that are looked at, at most

struct Segment {
    int req, qo0, rows, kv_len;
    int first, g, kv_lo, kv_end;
    int n_tiles, guard, all_see, whole;     // whole: written to o
    int64_t unit;                           // else: place of its first row's partial
    int64_t pad;
};

template <int D>
struct Lay {
    static constexpr int kSlots = D == 128 ? 3 : 6;
    static constexpr int kQBytes = kRows * D * 2, kTileBytes = kTok * D * 2;
    static constexpr int kSmemQ = 0, kSmemK = kQBytes, kSmemV = kSmemK + kSlots * kTileBytes, kSmemBar = kSmemV + kSlots * kTileBytes;
    // barriers
    static constexpr int kKFull = 0, kKEmpty = kSlots, kVFull = 2 * kSlots, kVEmpty = 3 * kSlots, kVRaw = 4 * kSlots, kVClean = 5 * kSlots;
    static constexpr int kSFull = 6 * kSlots, kPFull = kSFull + 2, kODone = kPFull + 2, kOEmpty = kODone + 2, kQFull = kOEmpty + 2;
    static constexpr int kQEmpty = kQFull + 1, kSegFull = kQEmpty + 1, kSegEmpty = kSegFull + kSegs, kBars = kSegEmpty + kSegs;
    static constexpr int kSmemSeg = kSmemBar + (kBars * 8 + 63) / 64 * 64;
    static constexpr int kBadWords = kGuarded * kTok / 32;
    static constexpr int kSmemBad = kSmemSeg + kSegs * static_cast<int>(sizeof(Segment));   // [kSegs][kBadWords + 1]: bits, then any
    static constexpr int kSmemMisc = kSmemBad + kSegs * (kBadWords + 1) * 4;                // tensor memory, abort
    static constexpr int kBytes = kSmemMisc + 8 + kThreads / 32 * 8 + 32 + 32 + 1024;       // sums, borders, entry; alignment slack
    static constexpr uint32_t kCols = 512;
    static_assert(sizeof(Segment) == 64 && kSmemMisc % 8 == 0 && kBytes <= 227 * 1024, "shared memory");
};

// Key tiles of an entry's kv head: one at least where it has rows (which are then
// written).
__device__ __forceinline__ int tiles_of(const ChunkEntry &e) { return e.q_len == 0 ? 0 : max(1, (e.kv_len + kTok - 1) / kTok); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
chunk_rows_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ Maps maps, const int box) {
    using bf16 = __nv_bfloat16;
    using L = Lay<D>;
    constexpr int S = L::kSlots, kChunks = D / 8;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t s_base = smem_u32(sm);
    long long *s_sum = reinterpret_cast<long long *>(sm + L::kSmemMisc + 8);           // a warp's tiles
    int(*s_at)[4] = reinterpret_cast<int(*)[4]>(sm + L::kSmemMisc + 8 + kThreads / 32 * 8);   // where the CTA's tiles begin and end:
                                                         // entry, head, tile, the item's tiles
    ChunkEntry *s_entry = reinterpret_cast<ChunkEntry *>(sm + L::kSmemMisc + 8 + kThreads / 32 * 8 + 32);
    Segment *segs = reinterpret_cast<Segment *>(sm + L::kSmemSeg);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + L::kSmemMisc + 4);
    auto bar = [&](int i) -> uint32_t { return s_base + L::kSmemBar + 8 * i; };
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int shift = p.group_shift, G = 1 << shift, HK = p.n_kv_heads, c = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    // ---- barriers, tensor memory
    if (tid == 0) {
        for (int i = 0; i < L::kBars; ++i) {
            uint32_t count = 1;
            if ((i >= L::kPFull && i < L::kODone) || (i >= L::kOEmpty && i < L::kQFull)) count = 4;
            else if (i >= L::kSegEmpty) count = 7;       // products, query tiles, V tiles, four softmax warps
            mbar_init(bar(i), count);
        }
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid == 32) asm volatile("prefetch.tensormap [%0];\nprefetch.tensormap [%1];\n" ::"l"(&maps.k), "l"(&maps.v) : "memory");
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(s_base + L::kSmemMisc), "r"(L::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    fence_before();
    // ---- this CTA's tiles: sums of the entries' tiles, a run of entries per thread
    long long n_all;                                     // tiles of all items
    int n;                                               // of this CTA
    {
        const int per = (p.batch + kThreads - 1) / kThreads, b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += tiles_of(load_chunk_entry(p, b, c == 0));
        long long inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        long long pre = inc - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) pre += s_sum[w];
            total += s_sum[w];
        }
        n_all = total * HK;
        const ChunkDeal deal{n_all, static_cast<int>(gridDim.x)};
        const bool mine_some = n_all > 0 && c < deal.parts();
        const long long x[2] = {mine_some ? deal.begin(c) : 0, mine_some ? deal.begin(c + 1) : 0};
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (x[k] >= pre * HK && x[k] < (pre + mine) * HK) {
                long long at = pre * HK;
                for (int b = b0; b < b1; ++b) {
                    const ChunkEntry e = load_chunk_entry(p, b, false);
                    const int t = tiles_of(e);
                    if (x[k] < at + static_cast<long long>(t) * HK) {
                        const long long in = x[k] - at;
                        s_at[k][0] = b;
                        s_at[k][1] = static_cast<int>(in / t);
                        s_at[k][2] = static_cast<int>(in % t);
                        s_at[k][3] = t;
                        if (k == 0) *s_entry = e;
                        break;
                    }
                    at += static_cast<long long>(t) * HK;
                }
            }
        __syncthreads();
        long long lo = x[0], hi = x[1];
        if (mine_some && !p.cut) {                       // whole items: those that begin in [lo, hi)
            if (s_at[0][2] > 0) lo += s_at[0][3] - s_at[0][2];
            if (hi < n_all && s_at[1][2] > 0) hi += s_at[1][3] - s_at[1][2];
        }
        n = static_cast<int>(hi - lo);                   // (a CTA's tiles are far fewer than 2^31)
    }
    fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(sm + L::kSmemMisc), 0);
    if (n <= 0) {
        if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(L::kCols));
        return;
    }
    auto give_up = [&](int code) {
        if (lane == 0 && *s_abort == 0) {
            *s_abort = 1;
            record_error(p.err, code);
        }
    };
    // use `i` of a ring of `places` barriers from `first` on: the wait for it to be full, or for its place to be free
    auto full = [&](int first, int places, int i) -> bool {
        return __all_sync(0xffffffffu, *s_abort == 0 && bar_wait(bar(first + i % places), (i / places) & 1));
    };
    auto empty = [&](int first, int places, int i) -> bool {
        return __all_sync(0xffffffffu, *s_abort == 0 && bar_wait(bar(first + i % places), ((i / places) & 1) ^ 1));
    };
    auto done_with = [&](int s) {                        // a segment's place in the ring, by a warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kSegEmpty + s % kSegs));
    };
    auto slot_at = [&](int req, int j) -> int {
        const int i = j / p.page_size, page = __ldg(p.req_to_page + static_cast<int64_t>(req) * p.max_pages + i);
        const bool ok = static_cast<unsigned long long>(static_cast<long long>(page)) < static_cast<unsigned long long>(p.n_pages);
        if (!ok) record_error(p.err, page);
        return (ok ? page : 0) * p.page_size + (j - i * p.page_size);
    };

    if (warp == 1) {
        // ================= the list of segments, and the copies
        int b = s_at[0][0], g = s_at[0][1], t0 = s_at[0][2], left = n, listed = 0;
        ChunkEntry e = *s_entry;
        int t_item = tiles_of(e);
        auto next_item = [&]() {
            t0 = 0;
            if (++g < HK) return;
            g = 0;
            for (t_item = 0; t_item == 0 && ++b < p.batch;) {      // 32 entries at a time, the first that has tiles
                const int mine = b + lane < p.batch ? tiles_of(load_chunk_entry(p, b + lane, false)) : 0;
                const unsigned some = __ballot_sync(0xffffffffu, mine > 0);
                if (!some) {
                    b += 31;
                    continue;
                }
                b += __ffs(some) - 1;
                e = load_chunk_entry(p, b, false);
                t_item = tiles_of(e);
            }
        };
        if (!p.cut && t0 > 0) next_item();
        auto list = [&]() -> bool {
            if (left == 0) return true;
            if (!empty(L::kSegEmpty, kSegs, listed)) return false;
            const int len = min(t_item - t0, left);
            Segment s;
            s.req = e.req, s.qo0 = e.qo0, s.rows = e.q_len << shift, s.kv_len = e.kv_len;
            s.first = e.first, s.g = g, s.kv_lo = t0 * kTok, s.kv_end = max(s.kv_lo, min(e.kv_len, (t0 + len) * kTok));
            s.n_tiles = len;
            s.all_see = min(chunk_limit(p, e, 0), s.kv_end - 1);
            s.guard = s.all_see < s.kv_lo ? 0 : (s.all_see + 1 - s.kv_lo) / kTok;
            s.whole = t0 == 0 && len == t_item;
            s.unit = (static_cast<int64_t>(c) + static_cast<int64_t>(b) * HK + g) * p.part_rows;
            if (lane == 0) {
                segs[listed % kSegs] = s;
                mbar_arrive(bar(L::kSegFull + listed % kSegs));
                if (p.cut) {                              // the CTAs of the item's first and last tile
                    const int64_t item = static_cast<int64_t>(b) * HK + g;
                    if (t0 == 0) p.cut[2 * item] = c;
                    if (t0 + len == t_item) p.cut[2 * item + 1] = c;
                }
            }
            __syncwarp();
            ++listed;
            left -= len;
            t0 += len;
            if (t0 == t_item && left > 0) next_item();
            return true;
        };
        const int per = box > 0 ? box : 4;
        const bool active = lane < kTok / per;
        auto fetch = [&](int s, int t, int (&row)[4]) {            // pool rows of this lane's part of a tile
            const Segment &q = segs[s % kSegs];
            const int j = q.kv_lo + t * kTok + lane * per, end = q.kv_end, req = q.req;
            if (!active) return;
            if (box > 0) {
                row[0] = j < end ? slot_at(req, j) : 0;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) row[u] = j + u < end ? slot_at(req, j + u) : 0;
            }
        };
        auto issue = [&](const CUtensorMap *map, uint32_t dst, uint32_t bar_full, const int (&row)[4], int head) {
            if (lane == 0) expect_bytes(bar_full, L::kTileBytes);
            __syncwarp();
            if (!active) return;
            if (box > 0) {
                copy_box(dst + lane * per * (D * 2), map, head * (D / 64), row[0] >> 3, bar_full);
            } else {
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    copy_rows4(dst + (lane >> 1) * (D * 16) + h * 1024 + (lane & 1) * 512, map, head * D + h * 64, row, bar_full);
            }
        };
        int s = 0, t = 0, plain = 0, raw = 0, done_k = 0;           // segment, tile in it; V tiles of either kind so far
        bool ok = true;
        int next[4] = {0, 0, 0, 0};
        ok = list();
        if (ok) fetch(0, 0, next);
        for (int i = 1; ok && i < kAhead; ++i) ok = list();
        for (int i = 0; ok && i < n; ++i) {
            const int row[4] = {next[0], next[1], next[2], next[3]};
            const int head = segs[s % kSegs].g, len = segs[s % kSegs].n_tiles, guard = segs[s % kSegs].guard;
            const bool look = t >= guard;
            if (++t == len) {
                t = 0;
                ++s;
                if (!list()) break;
            }
            if (i + 1 < n) fetch(s, t, next);
            if (!empty(L::kKEmpty, S, i)) break;
            issue(&maps.k, s_base + L::kSmemK + (i % S) * L::kTileBytes, bar(L::kKFull + i % S), row, head);
            done_k = i + 1;
            if (!empty(L::kVEmpty, S, i)) break;
            const int at = look ? L::kVRaw + raw++ % S : L::kVFull + plain++ % S;
            issue(&maps.v, s_base + L::kSmemV + (i % S) * L::kTileBytes, bar(at), row, head);
        }
        if (plain + raw < n) give_up(-5101);
        // no copy is in flight when the CTA ends, also after a wait that gave up
        for (int i = max(0, done_k - S); i < done_k; ++i) bar_wait(bar(L::kKFull + i % S), (i / S) & 1);
        for (int i = max(0, plain - S); i < plain; ++i) bar_wait(bar(L::kVFull + i % S), (i / S) & 1);
        for (int i = max(0, raw - S); i < raw; ++i) bar_wait(bar(L::kVRaw + i % S), (i / S) & 1);
    } else if (warp == 0) {
        // ================= products; S of tile t + 1 goes before P V of tile t
        const uint32_t id_s = idesc(kRows, kTok, 0), id_o = idesc(kRows, D, 1);
        const uint64_t dq = sdesc(s_base + L::kSmemQ, 16, D * 16), dk = sdesc(s_base + L::kSmemK, 16, D * 16);
        const uint64_t dv = sdesc(s_base + L::kSmemV, 1024, D * 16);
        const uint32_t hi = static_cast<uint32_t>(dq >> 32), v_hi = static_cast<uint32_t>(dv >> 32);
        const uint32_t q_lo = static_cast<uint32_t>(dq), k_lo = static_cast<uint32_t>(dk), v_lo = static_cast<uint32_t>(dv);
        auto commit = [&](int i) {
            if (elect()) mma_commit(bar(i));
        };
        auto full_fast = [&](int first, int places, int i) -> bool { return wait_fast(bar(first + i % places), (i / places) & 1); };
        int ss = 0, st = 0, sn = 0;                       // S: segment, tile in it, its tiles
        auto issue_s = [&](int i) -> bool {
            if (st == 0) {
                if (!full_fast(L::kSegFull, kSegs, ss)) return false;
                sn = segs[ss % kSegs].n_tiles;
                if (!full_fast(L::kQFull, 1, ss)) return false;
            }
            if (!full_fast(L::kKFull, S, i)) return false;
            fence_after();
            if (elect()) {
                const uint32_t qa = q_lo, ka = k_lo + (i % S) * (L::kTileBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_f16(tmem + (i & 1) * kTok, desc_at(qa + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), hi),
                            desc_at(ka + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), hi), id_s, ks > 0);
                mma_commit(bar(L::kSFull + (i & 1)));
                mma_commit(bar(L::kKEmpty + i % S));
            }
            if (++st == sn) {
                commit(L::kQEmpty);
                st = 0;
                ++ss;
            }
            return true;
        };
        int ps = 0, pt = 0, pn = 0, guard = 0, plain = 0, raw = 0;
        bool ok = issue_s(0);
        for (int i = 0; ok && i < n; ++i) {
            if (i + 1 < n && !issue_s(i + 1)) { ok = false; break; }
            if (pt == 0) {
                pn = segs[ps % kSegs].n_tiles;
                guard = segs[ps % kSegs].guard;
                if (!wait_fast(bar(L::kOEmpty + (ps & 1)), ((ps >> 1) & 1) ^ 1)) { ok = false; break; }
            }
            ok = pt < guard ? full_fast(L::kVFull, S, plain) : full_fast(L::kVClean, S, raw);
            if (pt < guard) ++plain;
            else ++raw;
            if (!ok || !full_fast(L::kPFull, 2, i)) { ok = false; break; }
            fence_after();
            if (elect()) {
                const uint32_t va = v_lo + (i % S) * (L::kTileBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < kTok / 16; ++ks)
                    mma_f16_ta(tmem + 256 + (ps & 1) * 128, tmem + (i & 1) * kTok + ks * 8, desc_at(va + ks * (2 * D * 16 >> 4), v_hi), id_o,
                               (pt > 0 || ks > 0) ? 1u : 0u);
                mma_commit(bar(L::kVEmpty + i % S));
                if (pt + 1 == pn) mma_commit(bar(L::kODone + (ps & 1)));
            }
            if (++pt == pn) {
                done_with(ps);
                pt = 0;
                ++ps;
            }
        }
        if (!ok) give_up(-5102);
        __syncwarp();
    } else if (warp == 2) {
        // ================= query tiles.  The maximum is of the products, so a scale
        // below 0 is taken into q, and one of 0 makes q 0.  Rows behind the
        // entry's are left as they are: their scores are read by nobody.
        const uint32_t q_and = p.scale_log2 == 0.f ? 0u : ~0u, q_xor = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        const bf16 *q = static_cast<const bf16 *>(p.q);
        for (int s = 0, i = 0; i < n; ++s) {
            if (!full(L::kSegFull, kSegs, s) || !empty(L::kQEmpty, 1, s)) { give_up(-5103); break; }
            const Segment &x = segs[s % kSegs];
            const int rows = x.rows, qo0 = x.qo0, g = x.g;
            i += x.n_tiles;
            unsigned char *dst = sm + L::kSmemQ;
            for (int u0 = lane; u0 < rows * kChunks; u0 += 32 * 16) {     // 16 chunks per lane on their way
                uint4 w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int u = u0 + 32 * k, r = u / kChunks, ch = u % kChunks;
                    if (u < rows * kChunks)
                        w[k] = *reinterpret_cast<const uint4 *>(
                            q + (static_cast<int64_t>(qo0 + (r >> shift)) * p.n_heads + g * G + (r & (G - 1))) * D + ch * 8);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int u = u0 + 32 * k, r = u / kChunks, ch = u % kChunks;
                    if (u >= rows * kChunks) break;
                    w[k].x = (w[k].x & q_and) ^ q_xor, w[k].y = (w[k].y & q_and) ^ q_xor;
                    w[k].z = (w[k].z & q_and) ^ q_xor, w[k].w = (w[k].w & q_and) ^ q_xor;
                    *reinterpret_cast<uint4 *>(dst + sw_at<D>(r, ch)) = w[k];
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kQFull));
            done_with(s);
        }
    } else if (warp == 3) {
        // ================= V tiles that not every row sees wholly
        int raw = 0;
        bool ok = true;
        for (int s = 0, i = 0; ok && i < n; ++s) {
            if (!full(L::kSegFull, kSegs, s)) { ok = false; break; }
            const Segment &x = segs[s % kSegs];
            uint32_t *bad = reinterpret_cast<uint32_t *>(sm + L::kSmemBad) + (s % kSegs) * (L::kBadWords + 1);
            if (x.guard < x.n_tiles)
                for (int w = lane; w <= L::kBadWords; w += 32) bad[w] = 0;
            __syncwarp();
            for (int t = x.guard; t < x.n_tiles; ++t, ++raw) {
                if (!full(L::kVRaw, S, raw)) { ok = false; break; }
                unsigned char *v = sm + L::kSmemV + ((i + t) % S) * L::kTileBytes;
                for (int r = lane; r < kTok; r += 32) {
                    const int j = x.kv_lo + t * kTok + r;
                    if (j <= x.all_see) continue;
                    if (j >= x.kv_end) {
                        for (int ch = 0; ch < kChunks; ++ch) *reinterpret_cast<uint4 *>(v + sw_at<D>(r, ch)) = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    bool found = false;
#pragma unroll 4
                    for (int ch = 0; ch < kChunks; ++ch) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(v + sw_at<D>(r, ch));
                        found |= not_finite(w.x) || not_finite(w.y) || not_finite(w.z) || not_finite(w.w);
                    }
                    if (found) {
                        for (int d = 0; d < D; ++d) {
                            uint16_t *y = reinterpret_cast<uint16_t *>(v + sw_at<D>(r, d / 8)) + (d & 7);
                            if ((*y & 0x7f80u) == 0x7f80u) *y = 0;
                        }
                        atomicOr(bad + ((t - x.guard) * kTok + r) / 32, 1u << (r & 31));
                        bad[L::kBadWords] = 1;
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kVClean + raw % S));
            }
            i += x.n_tiles;
            done_with(s);
        }
        if (!ok) give_up(-5104);
    } else {
        // ================= softmax and output: a row per thread
        const int row = tid & (kRows - 1);
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float sc = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
        bool ok = true;
        for (int s = 0, i0 = 0; ok && i0 < n; ++s) {
            if (!full(L::kSegFull, kSegs, s)) { ok = false; break; }
            const Segment x = segs[s % kSegs];
            const bool busy = (warp & 3) * 32 < x.rows;
            const int lim = row >= x.rows ? -1 : min(p.causal ? x.first + (row >> shift) : x.first, x.kv_len - 1);
            const uint32_t t_o = tmem + 256 + (s & 1) * 128 + lane_off;
            float m = -INFINITY, l = 0.f;
            for (int t = 0; t < x.n_tiles; ++t) {
                const int i = i0 + t;
                if (!full(L::kSFull, 2, i)) { ok = false; break; }
                if (!busy) {
                    if (lane == 0) mbar_arrive(bar(L::kPFull + (i & 1)));
                    continue;
                }
                fence_after();
                const uint32_t t_s = tmem + (i & 1) * kTok + lane_off;
                float sv[2][64];
                tmem_ld64(t_s, sv[0]);
                tmem_ld64(t_s + 64, sv[1]);
                auto v = [&](int u) -> float & { return sv[u >> 6][u & 63]; };
                const int j0 = x.kv_lo + t * kTok;
                if (j0 + kTok - 1 > lim) {
#pragma unroll
                    for (int u = 0; u < kTok; ++u)
                        if (j0 + u > lim) v(u) = -INFINITY;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int u = 0; u < kTok; u += 2) mx[(u >> 1) & 3] = max3(mx[(u >> 1) & 3], v(u), v(u + 1));
                const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                const bool raise = mt > m + kRescale || (m == -INFINITY && mt != -INFINITY);
                const bool touch = raise && t > 0 && m != -INFINITY;
                const float alpha = raise ? exp2f(m - mt) : 1.f;
                if (__any_sync(0xffffffffu, touch)) {
                    // P V of the tile before may still run
                    if (!full(L::kVEmpty, S, i - 1)) { ok = false; break; }
                    fence_after();
                    const float f = touch ? alpha : 1.f;
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        float y[32];
                        tmem_ld32(t_o + d, y);
#pragma unroll
                        for (int u = 0; u < 32; ++u) y[u] *= f;
                        tmem_st32(t_o + d, y);
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
                for (int d = 0; d < kTok; d += 16) {
                    uint32_t pk[8];
#pragma unroll
                    for (int u = 0; u < 16; u += 2) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(v(d + u), v(d + u + 1)), sc2, neg2), x0, x1);
                        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                        sum[(u >> 1) & 1] = f2_add(sum[(u >> 1) & 1], f2_pack(p0, p1));
                        const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                        pk[u >> 1] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    tmem_st8u(t_s + d / 2, pk);
                }
                float a0, a1, a2, a3;
                f2_unpack(sum[0], a0, a1);
                f2_unpack(sum[1], a2, a3);
                l += (a0 + a1) + (a2 + a3);
                asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kPFull + (i & 1)));
            }
            i0 += x.n_tiles;
            if (!ok || !full(L::kODone, 2, s)) { ok = false; break; }
            if (busy) {
                fence_after();
                const float inv = chunk_inverse(l, x.whole && lim >= 0);
                const uint32_t *bad = reinterpret_cast<const uint32_t *>(sm + L::kSmemBad) + (s % kSegs) * (L::kBadWords + 1);
                const bool some_bad = x.guard < x.n_tiles && *static_cast<const volatile uint32_t *>(bad + L::kBadWords) != 0;
                const int64_t at = (static_cast<int64_t>(x.qo0 + (row >> shift)) * p.n_heads + x.g * G + (row & (G - 1))) * D;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    __syncwarp();
                    float y[32];
                    tmem_ld32(t_o + d, y);
                    if (some_bad) {     // values that are not finite, for the rows that see them
                        for (int w = 0; w < L::kBadWords; ++w)
                            for (uint32_t bits = bad[w]; bits; bits &= bits - 1) {
                                const int j = x.kv_lo + x.guard * kTok + w * 32 + __ffs(bits) - 1;
                                if (j > lim) continue;
                                const bf16 *z = static_cast<const bf16 *>(p.v_buffer) +
                                                ((p.layer_row0 + slot_at(x.req, j)) * p.n_kv_heads + x.g) * D + d;
#pragma unroll
                                for (int u = 0; u < 32; ++u) {
                                    const float f = __bfloat162float(z[u]);
                                    if (!isfinite(f)) y[u] += f;
                                }
                            }
                    }
                    if (row >= x.rows) continue;
                    if (x.whole) {
#pragma unroll
                        for (int u = 0; u < 32; u += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(y[u + 2 * k] * inv, y[u + 2 * k + 1] * inv);
                                w[k] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            *reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.o) + at + d + u) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 32; u += 4)
                            *reinterpret_cast<float4 *>(p.o_part + (x.unit + row) * D + d + u) =
                                make_float4(y[u] * inv, y[u + 1] * inv, y[u + 2] * inv, y[u + 3] * inv);
                    }
                }
                if (!x.whole && row < x.rows) *reinterpret_cast<float2 *>(p.ml_part + 2 * (x.unit + row)) = make_float2(m, l);
                fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kOEmpty + (s & 1)));
            done_with(s);
        }
        if (!ok) give_up(-5105);
    }
    fence_before();
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(L::kCols));
}

// The join of the items that lie in several CTAs: a warp per row of an item.
template <int D>
__global__ void __launch_bounds__(kThreads) rows_join_kernel(const __grid_constant__ ChunkParams p, const int parts) {
    const int b = blockIdx.z, g = blockIdx.y, row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), G = 1 << p.group_shift;
    const ChunkEntry e = load_chunk_entry(p, b, false);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (row >= e.q_len << p.group_shift) return;
    const int64_t item = static_cast<int64_t>(b) * p.n_kv_heads + g;
    const int2 c = __ldcg(reinterpret_cast<const int2 *>(p.cut) + item);
    const int n = item_pieces(c.x, c.y, parts);           // (several tiles: every row sees some position)
    if (n == 0) return;
    const int64_t unit = (c.x + item) * p.part_rows + row;
    join_row<__nv_bfloat16, D>(p, n, [&](int s) { return unit + static_cast<int64_t>(s) * p.part_rows; },
                               (static_cast<int64_t>(e.qo0 + (row >> p.group_shift)) * p.n_heads + g * G + (row & (G - 1))) * D);
}

template <int D>
cudaError_t run(const ChunkParams &p, int parts, int group, cudaStream_t s) {
    using L = Lay<D>;
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        e = cudaFuncSetAttribute(chunk_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (e != cudaSuccess) return e;
        attr_done.fetch_or(bit);
    }
    const int box = box_rows(p.page_size, kTok);
    Maps maps;
    if (!pool_maps(&maps, p, D, box)) return cudaErrorInvalidValue;
    chunk_rows_kernel<D><<<parts, kThreads, L::kBytes, s>>>(p, maps, box);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.cut) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.max_q_len * group + kThreads / 32 - 1) / (kThreads / 32), p.n_kv_heads, p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_join_kernel<D>, p, parts);
}

}  // namespace

cudaError_t launch_chunk_rows(const ChunkParams &p, int parts, int head_dim, int group, cudaStream_t s) {
    return head_dim == 128 ? run<128>(p, parts, group, s) : run<64>(p, parts, group, s);
}

}  // namespace pkv
