// Device helpers shared by the attention kernels: the tiles a sequence's rows see, paged TMA loads.
#pragma once

#include "dev_common.cuh"
#include "layer_internal.h"

namespace lora {
namespace dev {

// The cache tiles of `tk` tokens that the rows of one sequence (or some of its rows) see: first the
// tiles with sinks (s_tiles of them, from token 0), then those from lo_tile to the last token.
struct TileRange {
    int len;        // tokens in the cache that the rows may see: one past the last row's position
    int first;      // position of the first row (negative: rows before the sequence's start see nothing)
    int s_tiles, lo_tile, n;
};
__device__ __forceinline__ TileRange tile_range(int first, int last, int window, int sinks, int tk) {
    TileRange r;
    r.first = first;
    r.len = last + 1;
    const int lo = window ? max(0, first - window + 1) : 0;
    r.lo_tile = lo / tk;
    r.s_tiles = min((min(sinks, lo) + tk - 1) / tk, r.lo_tile);
    r.n = last < 0 ? 0 : r.s_tiles + (last / tk + 1 - r.lo_tile);
    return r;
}
__device__ __forceinline__ int tile_token(const TileRange& r, int i, int tk) {
    return (i < r.s_tiles ? i : r.lo_tile + i - r.s_tiles) * tk;
}
// Tokens of sequence s, clamped to what its page table can hold.
__device__ __forceinline__ int cache_len(const CacheView& c, int s) {
    return (int)min((long long)max(c.kv_lens[s], 0), (long long)c.pages_per_seq * c.page_size);
}

// 4-D tiled load of one granule of one head's 64 features. The tensor map's axes past the features
// are ordered by stride, so the coordinates come in the map's order.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
// order packs which coordinate (0 head, 1 token, 2 page) each of the map's axes 1..3 takes, 2 bits each.
__device__ __forceinline__ void tma_load_kv(uint32_t dst, const CUtensorMap* map, uint32_t bar, int order, int feature, int head,
                                            int token, int page) {
    const int a = order & 3, b = (order >> 2) & 3, c = order >> 4;
    tma_load_4d(dst, map, bar, feature, a == 0 ? head : a == 1 ? token : page, b == 0 ? head : b == 1 ? token : page,
                c == 0 ? head : c == 1 ? token : page);
}
__device__ __forceinline__ void fence_proxy_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 2^x by the hardware's instruction (x = -inf gives 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace dev
}  // namespace lora
