// pkv_chunk.cuh -- what the kernels of the chunk attention share (internal).
#pragma once

#include "pkv_common.cuh"
#include "pkv_launch.h"

namespace pkv {

// Entry b's rows of q and its context, checked: an entry with an error has no
// rows.  first = position that its first row sees up to (causal), below 0 if
// that row sees nothing.
struct ChunkEntry {
    int req, qo0, q_len, kv_len, first;
};

__device__ __forceinline__ ChunkEntry load_chunk_entry(const ChunkParams &p, int b, bool report) {
    ChunkEntry e;
    e.req = __ldg(p.req_pool_indices + b);
    e.qo0 = __ldg(p.qo_indptr + b);
    const int end = __ldg(p.qo_indptr + b + 1);
    e.kv_len = __ldg(p.seq_lens + b);
    const long long q_len = static_cast<long long>(end) - e.qo0;
    e.q_len = static_cast<int>(q_len);
    bool ok = true;
    int bad = 0;
    if (static_cast<unsigned>(e.req) >= static_cast<unsigned>(p.num_reqs)) ok = false, bad = e.req;
    else if (e.qo0 < 0 || end > p.n_q || q_len < 0) ok = false, bad = e.qo0 < 0 || e.qo0 > p.n_q ? e.qo0 : end;
    else if (q_len > p.max_q_len) ok = false, bad = e.q_len;
    else if (static_cast<unsigned>(e.kv_len) > static_cast<unsigned>(p.max_len)) ok = false, bad = e.kv_len;
    if (!ok) {
        if (report) record_error(p.err, bad);
        e.req = e.qo0 = e.q_len = e.kv_len = 0;
    }
    e.first = p.causal ? e.kv_len - e.q_len : e.kv_len - 1;
    return e;
}

// The entry that lane `from` holds, by a whole warp: values that are then known to be
// one for all lanes, so that branches on them take no care of lanes that part (4 x 2048
// tokens at 8K to 16K: 914 us, 984 without; in fp32 4 x 512 at 2K 1060 and 1084).
__device__ __forceinline__ ChunkEntry entry_of_lane(ChunkEntry e, int from) {
    e.req = __shfl_sync(0xffffffffu, e.req, from), e.qo0 = __shfl_sync(0xffffffffu, e.qo0, from);
    e.q_len = __shfl_sync(0xffffffffu, e.q_len, from), e.kv_len = __shfl_sync(0xffffffffu, e.kv_len, from);
    e.first = __shfl_sync(0xffffffffu, e.first, from);
    return e;
}

// The entry that the CTAs of grid z take, by a whole warp: among 32 neighbouring ones
// that of the z-th longest context, so that the short ones fill the gaps at the end.
// (16 chunks of up to 448 tokens over up to 1500 states 37.9 us, in their own order
// 41.5; 4 x 2048 tokens at 8K to 16K 792 and 804 at head_dim 64, 914 either way at
// 128; entries of one length pay for the look at all 32: 8 prompts of 2048 tokens
// 275 us, 271 in their own order.)
// report: the warp of grid z looks at all 32 (one does for each 32).
__device__ __forceinline__ ChunkEntry load_longest_entry(const ChunkParams &p, int z, bool report) {
    const int lane = threadIdx.x & 31, b = (z & ~31) + lane, at = z & 31;
    ChunkEntry e = load_chunk_entry(p, min(b, p.batch - 1), report && at == 0 && b < p.batch);
    const int len = b >= p.batch ? -2 : e.q_len == 0 ? -1 : e.kv_len;
    int longer = 0;                                    // entries before this one
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const int other = __shfl_sync(0xffffffffu, len, j);
        longer += other > len || (other == len && j < lane);
    }
    return entry_of_lane(e, __ffs(__ballot_sync(0xffffffffu, longer == at)) - 1);
}

// last position that the row at place i of its entry sees
__device__ __forceinline__ int chunk_limit(const ChunkParams &p, const ChunkEntry &e, int i) {
    return p.causal ? e.first + i : e.first;
}

// What a row's weighted sum of values is multiplied by, l being the sum of its weights:
// 0 for a row that sees nothing, NaN (0 / 0) for one whose scores are all -inf.
__device__ __forceinline__ float chunk_inverse(float l, bool sees) { return l == 0.f ? (sees ? NAN : 0.f) : 1.f / l; }

// the partial sums of split `split`: row `row` of q, head `head`
__device__ __forceinline__ int64_t chunk_unit(const ChunkParams &p, int split, int row, int head) {
    return (static_cast<int64_t>(split) * p.n_q + row) * p.n_heads + head;
}

}  // namespace pkv
