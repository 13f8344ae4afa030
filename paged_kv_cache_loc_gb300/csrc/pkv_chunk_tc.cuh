// pkv_chunk_tc.cuh -- what the tensor-core kernels of the chunk attention share:
// tiles in shared memory, TMA copies of pages, waits (internal).
#pragma once

#include <cuda.h>

#include "pkv_chunk.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kRescale = 8;                 // the reference is raised by 2^8 at least

// Byte offset of 16-byte chunk ch of row r in a tile: eight rows at a time, their
// 64-column halves as 8 x 128 bytes one after the other, chunk c of a row at c ^
// (r % 8).  So a run of rows of a page is one box of the tensor map, and the
// steps between groups of rows (D * 16 bytes) and halves (1024) are those of a
// matrix descriptor.
template <int D>
__device__ __forceinline__ uint32_t sw_at(int r, int ch) {
    return (r >> 3) * (D * 16) + (ch >> 3) * 1024 + (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// One lane of a whole warp.  (With `lane == 0` instead the compiler does not know
// that one thread issues the asynchronous instructions behind it, and each costs
// several times as much.)
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
// TMA copies of a box of rows, or of four rows, to this CTA.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int half, int group, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(map), "r"(0), "r"(half), "r"(group), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy_rows4(uint32_t dst, const CUtensorMap *map, int x, const int (&row)[4], uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
        "[%7];\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
        : "memory");
}

// bar_wait of the warp that issues the products, with one answer for all lanes:
// what is done already, as it mostly is, costs one test that falls through.
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity) { return bar_wait(bar, parity); }
__device__ __forceinline__ bool wait_fast(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__builtin_expect(__all_sync(0xffffffffu, ok != 0), 1)) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity));
}

struct Maps {
    CUtensorMap k, v;
};

// Whether a word of two bf16 holds a value that is not finite.
__device__ __forceinline__ bool not_finite(uint32_t w) {
    const uint32_t e = w & 0x7f807f80u;
    return (e & 0xffffu) == 0x7f80u || (e >> 16) == 0x7f80u;
}

// The maps of a layer's K and V for boxes of `box` rows of a page (0: single rows,
// gathered four at a time).  Host.
bool pool_maps(Maps *maps, const ChunkParams &p, int D, int box);

// Rows of a page that a box may take: the largest power of two in page_size, `most`
// at most; below a swizzle atom of eight rows 0.
inline int box_rows(int page_size, int most) {
    int box = page_size & -page_size;
    if (box > most) box = most;
    return box < 8 ? 0 : box;
}

}  // namespace pkv
