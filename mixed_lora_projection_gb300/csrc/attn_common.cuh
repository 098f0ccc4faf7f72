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

// Zeros in place of the values of tokens [from, to) of a piece of TOK tokens in chunks of 64 features, where they
// are one run of bytes each, by n threads of which this is `me`. It is for tokens that no row sees (past the last
// one, or between the sinks and the window): they may hold anything, and their weight of 0 needs them finite. The
// caller fences. (One st.bulk a chunk took as long: a 16,384-token prompt with a window of 4,096, heads of 256, 999 us
// either way.)
template <int D, int TOK>
__device__ __forceinline__ void zero_tokens(uint32_t piece, int from, int to, int me, int n) {
    from = max(from, 0);
    to = min(to, TOK);
#pragma unroll 1
    for (int i = me; i < (to - from) * 8; i += n)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(piece + c * (TOK * 128) + from * 128 + i * 16), "r"(0)
                         : "memory");
}

// 2^x by the hardware's instruction (x = -inf gives 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One row of a split unit, by 128 threads: parts [0, n) with maximum and sum part_ml[at(c)] and
// unnormalised sums part_o[at(c)][D]. The four warps take every fourth part in one pass (a part's sums are
// loaded with its maximum, not after it), then add up; the order is the same in every run.
template <int D, class At>
__device__ __forceinline__ void join_row(const float* part_o, const float2* part_ml, int n, At at, __nv_bfloat16* out) {
    constexpr int E = D / 32;
    __shared__ float acc[4][D];
    __shared__ float2 ml[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int c = warp; c < n; c += 4) {
        const long long i = at(c);
        const float2 x = part_ml[i];
        float2 v[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) v[e] = *reinterpret_cast<const float2*>(part_o + i * D + lane * E + 2 * e);
        const float mn = fmaxf(m, x.x), ms = mn == -INFINITY ? 0.f : mn, w = ex2(x.x - ms), old = ex2(m - ms);
        m = mn;
        l = l * old + x.y * w;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            o[2 * e] = o[2 * e] * old + v[e].x * w;
            o[2 * e + 1] = o[2 * e + 1] * old + v[e].y * w;
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[warp][lane * E + e] = o[e];
    if (lane == 0) ml[warp] = make_float2(m, l);
    __syncthreads();
    m = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
    const float ms = m == -INFINITY ? 0.f : m;
    float w[4];
    l = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w[k] = ex2(ml[k].x - ms);
        l += ml[k].y * w[k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = threadIdx.x; e < D; e += 128)
        out[e] = __float2bfloat16_rn((acc[0][e] * w[0] + acc[1][e] * w[1] + acc[2][e] * w[2] + acc[3][e] * w[3]) * inv);
    __syncthreads();                     // before the next row's sums
}

}  // namespace dev
}  // namespace lora
