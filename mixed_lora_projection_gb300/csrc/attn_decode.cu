// Attention of a few new rows per sequence over the paged cache (at most 16 rows per key/value head:
// q_len x query heads per key/value head).
//
// The work is one pass over K and V, so it is bound by memory. All cache tiles of the call (64 or 128
// tokens of one head), sequence after sequence and head after head, form one line that is cut into
// equal parts, one per block: uneven lengths and few sequences fill the GPU alike. A block's part
// may end inside a unit (one head of one sequence); what it has then, unnormalised sums o with their
// running maximum m and sum l per row, goes to the workspace, and a second small kernel joins a
// unit's parts c in their order: M = max m_c, o = sum 2^(m_c - M) o_c / sum 2^(m_c - M) l_c.
//
// A block is four consumer warps and a TMA producer warp with a ring of K and V tiles. Per tile each
// consumer computes the scores of a quarter of the tokens (mma.sync m16n8k16: rows are padded to 16), the warps
// exchange row maxima, write the weights to shared memory as bf16 (the product with V takes bf16
// operands; their sum is kept of the unrounded fp32 weights) and each adds a quarter of the features
// of the product with V. With 16 rows the matrix work is a fraction of the loads' time, so the
// warp-level instruction serves, at two blocks per SM; more rows go to the prompt kernel, whose
// tcgen05 tiles of 128 rows the warp-level instruction cannot follow (six sequences with 48 rows
// per head of 256: 119 us here with three row tiles, 72 there, where one pass over the cache takes 41).
//
// Measured (one GB300): six chats of 3,000 to 32,768 tokens, 24 / 12 heads of 256, 221 us = 0.88 of the
// measured copy rate; 64 chats of 700 to 15,820 tokens, 48 / 8 heads of 128, 360 us = 0.89; 64 of 700 to
// 7,000 tokens, 16 heads of 64, 191 us = 0.78; one chat of 517 tokens 8 us with the join, by latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_common.cuh"

namespace lora {
namespace {

using namespace dev;

// Tokens of a tile. A tile costs the consumers' chain of waits and products (~1 us) whatever it holds, so
// heads of 64, whose tokens are few bytes, take twice as many (64 sequences of 700 to 7,000 tokens, 16
// heads of 64: 215 us with 64 tokens, 209 with 128).
template <int D>
constexpr int kTile = D == 64 ? 128 : 64;
constexpr int kConsumers = 128;
constexpr int kDecodeThreads = 160;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// First flat tile of block c of g: the line of w tiles cut into g equal parts.
__device__ __forceinline__ unsigned long long part_begin(unsigned long long w, unsigned g, unsigned c) { return w * c / g; }
// The block that flat tile t belongs to.
__device__ __forceinline__ unsigned part_of(unsigned long long w, unsigned g, unsigned long long t) {
    return (unsigned)(((t + 1) * g - 1) / w);
}

// Shared memory: Q rows, weights, row maxima and sums, prefix, barriers, then the ring (1024-aligned).
template <int D>
struct Layout {
    static constexpr int kRows = kDecodeRows, kTk = kTile<D>;
    static constexpr int kQStride = D + 8, kPStride = kTk + 8;   // padded rows: conflict-free ldmatrix
    static constexpr int kP = kRows * kQStride * 2;
    static constexpr int kMax = kP + kRows * kPStride * 2;
    static constexpr int kSum = kMax + 4 * kRows * 4;
    static constexpr int kBars = kSum + 4 * kRows * 4;           // full[slots], empty[slots] (16 at most each)
    static constexpr int kAbort = kBars + 32 * 8;
    static constexpr int kPrefix = kAbort + 16;                  // tiles before each sequence, then the sequences' lengths
    static constexpr int kSlot = kTk * D * 2;
};

// Where a block's walk over its part is: a piece of one unit at a time.
struct Walk {
    unsigned long long at, end;
    int i;               // sequence of the list
};

template <int D, int N>
__global__ void __launch_bounds__(kDecodeThreads, 2)
    decode_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ SeqList<N> list) {
    using S = Layout<D>;
    constexpr int kRows = S::kRows, kTk = S::kTk, kOwn = kTk / 4;        // kOwn: tokens of a consumer warp
    extern __shared__ __align__(1024) uint8_t raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* full = reinterpret_cast<uint64_t*>(raw + S::kBars);
    uint64_t* empty = full + 16;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(raw + S::kAbort);
    uint32_t* prefix = reinterpret_cast<uint32_t*>(raw + S::kPrefix);
    int* lens = reinterpret_cast<int*>(prefix + list.n + 1);
    const uint32_t ring = (smem_addr(raw + S::kPrefix + (2 * list.n + 1) * 4) + 1023u) & ~1023u;
    const int slots = p.slots;

    if (tid == 0) {
        for (int s = 0; s < slots; ++s) {
            mbar_init(smem_addr(&full[s]), 1);
            mbar_init(smem_addr(&empty[s]), 4);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    // tiles of one head before each sequence
    const AttnParams& a = p.a;
    griddep_wait();
    for (int i = tid; i < list.n; i += kDecodeThreads) {
        const int len = lens[i] = cache_len(a.c, list.seq[i]);
        prefix[i + 1] = (uint32_t)tile_range(len - list.q_len[i], len - 1, a.window, a.sinks, kTk).n;
    }
    __syncthreads();
    if (warp == 0) {
        uint32_t carry = 0;
        for (int i0 = 0; i0 < list.n; i0 += 32) {
            uint32_t v = i0 + lane < list.n ? prefix[i0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (i0 + lane < list.n) prefix[i0 + lane + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) prefix[0] = 0;
    }
    __syncthreads();
    const int n_kv = a.c.n_kv;
    const unsigned long long total = (unsigned long long)prefix[list.n] * n_kv;
    const unsigned grid = (unsigned)min((unsigned long long)gridDim.x, total);     // blocks that get a part
    if (blockIdx.x == 0)
        for (int i = tid; i <= list.n; i += kDecodeThreads) p.prefix[i] = prefix[i];
    griddep_launch_dependents();
    // sequences without a visible token: zeros
    for (int i = blockIdx.x; i < list.n; i += gridDim.x)
        if (prefix[i + 1] == prefix[i]) {
            const int per = n_kv * p.group * (D / 8);
            for (int v = tid; v < list.q_len[i] * per; v += kDecodeThreads) {
                const int row = list.row[i] + v / per, hq = v % per / (D / 8), c = v % (D / 8);
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * a.o_stride + hq * a.o_head + c * 8) =
                    make_uint4(0, 0, 0, 0);
            }
        }
    if (blockIdx.x >= grid) return;
    Walk w;
    w.at = part_begin(total, grid, blockIdx.x);
    w.end = part_begin(total, grid, blockIdx.x + 1);
    {
        int lo = 0, hi = list.n - 1;     // the last sequence that begins at or before the first tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((unsigned long long)prefix[mid] * n_kv <= w.at) lo = mid; else hi = mid - 1;
        }
        w.i = lo;
    }
    const uint64_t limit = a.wait_limit_ns;

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        const int chunks = D / 64, boxes = (kTk / p.granule) * chunks;
        const int gi = lane / chunks, ch = lane % chunks;
        const uint32_t box_bytes = (uint32_t)p.granule * 128;
        int slot = 0, issued = 0, allowed = a.debug_stall ? a.debug_stall - 1 : kNoStall;    // tiles until a test's stall
        uint32_t phase = 0;
        bool ok = true;
        while (ok && w.at < w.end) {
            const uint32_t nt = prefix[w.i + 1] - prefix[w.i];
            if (nt == 0) {
                ++w.i;
                continue;
            }
            const unsigned long long rel = w.at - (unsigned long long)prefix[w.i] * n_kv;
            const int head = (int)(rel / nt), t0 = (int)(rel % nt);
            const int t1 = (int)min((unsigned long long)nt, t0 + (w.end - w.at));
            const int s = list.seq[w.i], len = lens[w.i];
            const TileRange r = tile_range(len - list.q_len[w.i], len - 1, a.window, a.sinks, kTk);
            const int32_t* table = a.c.table + s * a.c.table_stride;
            // this lane's granule of tile t: its page (one past the last: zeros) and token in it
            auto place = [&](int t, int& page, int& tok) {
                const int j = tile_token(r, t, kTk) + gi * p.granule;
                page = -1;
                tok = 0;
                if (lane < boxes && j < len) {
                    const int pg = j / a.c.page_size;
                    page = table[pg];
                    tok = j - pg * a.c.page_size;
                    if (page < 0 || page >= a.c.n_pages) page = a.c.n_pages;
                }
            };
            int page, tok;
            place(t0, page, tok);
            const int t_stop = min(t1, t0 + allowed);
            if (a.debug_stall) allowed -= t_stop - t0;
            for (int t = t0; t < t_stop && ok; ++t) {
                int npage = -1, ntok = 0;
                if (t + 1 < t1) place(t + 1, npage, ntok);       // the next tile's pages, ahead of its turn
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, page >= 0)) * box_bytes;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (!wait_warp(smem_addr(&empty[slot]), phase ^ 1, abort_flag, a.status, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_addr(&full[slot]);
                    mbar_arrive_expect_tx(bar, bytes, lane == 0);
                    __syncwarp();
                    if (page >= 0)
                        tma_load_kv(ring + (uint32_t)slot * S::kSlot + (uint32_t)ch * (kTk * 128) + (uint32_t)gi * box_bytes,
                                    kv ? &p.tm_v : &p.tm_k, bar, kv ? p.v_order : p.k_order, ch * 64, head, tok, page);
                    ++issued;
                    if (++slot == slots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                page = npage;
                tok = ntok;
            }
            ok = ok && t_stop == t1;
            w.at += t1 - t0;
            if ((unsigned long long)prefix[w.i + 1] * n_kv <= w.at) ++w.i;
        }
        // The copies in flight land before the block may end, whoever gave up: consumers that did wait for none.
        if (lane == 0)
            for (int k = max(0, issued - slots); k < issued; ++k)
                wait_bounded(smem_addr(&full[k % slots]), (uint32_t)((k / slots) & 1), abort_flag, a.status, limit, false);
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int gr = lane >> 2, gc = lane & 3;
    const uint32_t q_base = smem_addr(raw), p_base = smem_addr(raw + S::kP);
    float* smax = reinterpret_cast<float*>(raw + S::kMax);
    float* ssum = reinterpret_cast<float*>(raw + S::kSum);
    const int g = p.group;
    int slot = 0;
    uint32_t phase = 0;
    // After a wait that ran out a warp runs on without data, so that the warps' barriers stay matched; the status
    // word says that the output is incomplete. It frees no slot any more: what it did not wait for may still be in
    // flight, and the producer would load over it.
    bool ok = true;
    while (w.at < w.end) {
        const uint32_t nt = prefix[w.i + 1] - prefix[w.i];
        if (nt == 0) {
            ++w.i;
            continue;
        }
        const unsigned long long rel = w.at - (unsigned long long)prefix[w.i] * n_kv;
        const int head = (int)(rel / nt), t0 = (int)(rel % nt);
        const int t1 = (int)min((unsigned long long)nt, t0 + (w.end - w.at));
        const int q_len = list.q_len[w.i], len = lens[w.i];
        const TileRange r = tile_range(len - q_len, len - 1, a.window, a.sinks, kTk);
        const int rows = q_len * g;
        // this unit's queries: through shared memory into the fragments of the score products
        for (int v = tid; v < kRows * (D / 8); v += kConsumers) {
            const int row = v / (D / 8), c = v % (D / 8);
            uint4 val = make_uint4(0, 0, 0, 0);
            if (row < rows) {
                const int qi = row / g, hq = head * g + row - qi * g;
                val = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                      (list.row[w.i] + qi) * a.q_stride + hq * a.q_head + c * 8);
            }
            *reinterpret_cast<uint4*>(raw + row * S::kQStride * 2 + c * 16) = val;
        }
        int pos[2];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[D / 32][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) pos[h] = gr + 8 * h < rows ? r.first + (gr + 8 * h) / g : -1;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        consumer_sync();
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            ldsm4(q_base + (uint32_t)((lane & 7) + ((lane >> 3) & 1) * 8) * (S::kQStride * 2) + (lane >> 4) * 16 + kk * 32, qf[kk]);

        for (int t = t0; t < t1; ++t) {
            const int j0 = tile_token(r, t, kTk);
            // ---- scores of this warp's tokens, in two chains of products
            float sc[2][kOwn / 8][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int n = 0; n < kOwn / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[x][n][e] = 0.f;
            ok = ok && wait_warp(smem_addr(&full[slot]), phase, abort_flag, a.status, limit);
            {
                const int tok = warp * kOwn + (lane & 7) + ((lane >> 4) & 1) * 8;
                const uint32_t krow = ring + (uint32_t)slot * S::kSlot + (uint32_t)tok * 128;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int n = 0; n < kOwn / 16; ++n) {
                        uint32_t b[4];
                        const int idx = (kk & 3) * 2 + ((lane >> 3) & 1);
                        ldsm4(krow + (kk >> 2) * (kTk * 128) + n * (16 * 128) + ((idx ^ (tok & 7)) << 4), b);
                        mma16816(sc[kk & 1][2 * n], qf[kk], b[0], b[1]);
                        mma16816(sc[kk & 1][2 * n + 1], qf[kk], b[2], b[3]);
                    }
            }
            const int kslot = slot;
            if (++slot == slots) {
                slot = 0;
                phase ^= 1;
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < kOwn / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + warp * kOwn + n * 8 + gc * 2 + (e & 1), ps = pos[e >> 1];
                    float x = (sc[0][n][e] + sc[1][n][e]) * a.scale_log2;
                    const bool seen = j <= ps && (a.window == 0 || j > ps - a.window || j < a.sinks);
                    x = seen ? x : -INFINITY;
                    sc[0][n][e] = x;
                    mx[e >> 1] = fmaxf(mx[e >> 1], x);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                if (gc == 0) smax[warp * kRows + gr + 8 * h] = mx[h];
            }
            consumer_sync();
            if (ok && lane == 0) mbar_arrive(smem_addr(&empty[kslot]));
            // ---- weights
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = gr + 8 * h;
                float mn = m[h];
#pragma unroll
                for (int x = 0; x < 4; ++x) mn = fmaxf(mn, smax[x * kRows + row]);
                const float ms = mn == -INFINITY ? 0.f : mn;
                const float alpha = ex2(m[h] - ms);
                m[h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < kOwn / 8; ++n) {
                    const float w0 = ex2(sc[0][n][2 * h] - ms), w1 = ex2(sc[0][n][2 * h + 1] - ms);
                    sum += w0 + w1;
                    *reinterpret_cast<uint32_t*>(raw + S::kP + row * S::kPStride * 2 + (warp * kOwn + n * 8 + gc * 2) * 2) =
                        pack_bf16x2(w0, w1);
                }
                l[h] = l[h] * alpha + sum;
                if (alpha != 1.f) {
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) {
                        o[n][2 * h] *= alpha;
                        o[n][2 * h + 1] *= alpha;
                    }
                }
            }
            ok = ok && wait_warp(smem_addr(&full[slot]), phase, abort_flag, a.status, limit);
            const uint32_t vt = ring + (uint32_t)slot * S::kSlot;
            // tokens that no row sees: past the last one, or in the sinks' last tile and the window's first
            if (r.len - j0 < kTk) {
                zero_tokens<D, kTk>(vt, r.len - j0, kTk, tid, kConsumers);
                fence_proxy_async_shared();
            }
            if (a.window && (unsigned)(t + 1 - r.s_tiles) < 2) {
                zero_tokens<D, kTk>(vt, a.sinks - j0, r.len - list.q_len[w.i] - a.window + 1 - j0, tid, kConsumers);
                fence_proxy_async_shared();
            }
            consumer_sync();
            // ---- product with V: this warp's quarter of the features
            {
                const int tok = (lane & 7) + ((lane >> 3) & 1) * 8;
                const uint32_t prow = p_base + (uint32_t)tok * (S::kPStride * 2) + (lane >> 4) * 16;
#pragma unroll
                for (int kt = 0; kt < kTk / 16; ++kt) {
                    uint32_t pa[4];
                    ldsm4(prow + kt * 32, pa);
                    const uint32_t vrow = vt + (uint32_t)(kt * 16 + tok) * 128;
#pragma unroll
                    for (int np = 0; np < D / 64; ++np) {
                        uint32_t b[4];
                        const int dv = warp * (D / 32) + np * 2 + (lane >> 4);
                        ldsm4t(vrow + (dv >> 3) * (kTk * 128) + (((dv & 7) ^ (tok & 7)) << 4), b);
                        mma16816(o[2 * np], pa, b[0], b[1]);
                        mma16816(o[2 * np + 1], pa, b[2], b[3]);
                    }
                }
            }
            // The slot's next load comes by TMA, which does not queue behind this warp's: they are done before it is freed.
            // (Without the fence, their results not yet used, the last loads of V read the next tile of K now and then:
            // heads of 256, whose ring has three slots, other bits in 1 of 1.4 million runs of random batches, and in 15
            // of 4,000 where a slow st.bulk kept a warp's loads waiting; with it none in 16,000 of those. It costs nothing
            // that shows: 64 chats of heads of 128 371 us, six of 256 221, either way.)
            __threadfence_block();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(smem_addr(&empty[slot]));
            if (++slot == slots) {
                slot = 0;
                phase ^= 1;
            }
        }

        // ---- the piece's end: the warps' sums of weights together
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x = l[h];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (gc == 0) ssum[warp * kRows + gr + 8 * h] = x;
        }
        consumer_sync();
        const bool whole = t0 == 0 && t1 == (int)nt;
        const long long part = 2ll * blockIdx.x + (t0 == 0 ? 1 : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = gr + 8 * h;
            if (row >= rows) continue;
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) sum += ssum[x * kRows + row];
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int qi = row / g, hq = head * g + row - qi * g;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (list.row[w.i] + qi) * a.o_stride + hq * a.o_head +
                                     warp * (D / 4) + gc * 2;
#pragma unroll
                for (int n = 0; n < D / 32; ++n)
                    *reinterpret_cast<uint32_t*>(out + n * 8) = pack_bf16x2(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
            } else {
                float* po = p.part_o + (part * kRows + row) * D + warp * (D / 4) + gc * 2;
#pragma unroll
                for (int n = 0; n < D / 32; ++n) *reinterpret_cast<float2*>(po + n * 8) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
                if (warp == 0 && gc == 0) p.part_ml[part * kRows + row] = make_float2(m[h], sum);
            }
        }
        w.at += t1 - t0;
        if ((unsigned long long)prefix[w.i + 1] * n_kv <= w.at) ++w.i;
    }
}

// Joins the parts of split units: a block takes one row of a unit at a time. (Joined by the block that
// ends last instead, in the same launch, one chat's step took 12.3 us against 10.3: one block then reads
// what four warps per row read at once.)
template <int D, int N>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ SeqList<N> list) {
    const AttnParams& a = p.a;
    const int g = p.group, most = p.most_rows, per = a.c.n_kv * most;
    for (int x = blockIdx.x; x < list.n * per; x += gridDim.x) {
        const int i = x / per, head = (x - i * per) / most, row = x - i * per - head * most, rows = list.q_len[i] * g;
        const int qi = row / g, hq = head * g + row - qi * g;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (list.row[i] + qi) * a.o_stride + hq * a.o_head;
        if (x == (int)blockIdx.x) {      // what the parameters tell is worked out first (one chat 8.9 -> 8.1 us)
            griddep_wait();
            griddep_launch_dependents();
        }
        const uint32_t all = p.prefix[list.n], p0 = p.prefix[i], nt = p.prefix[i + 1] - p0;
        if (row >= rows || nt == 0) continue;           // of units without tiles the first launch wrote the zeros
        const unsigned long long total = (unsigned long long)all * a.c.n_kv;
        const unsigned grid = (unsigned)min((unsigned long long)p.grid, total);
        const unsigned long long first = (unsigned long long)p0 * a.c.n_kv + (unsigned long long)head * nt;
        const unsigned c0 = part_of(total, grid, first), c1 = part_of(total, grid, first + nt - 1);
        if (c0 == c1) continue;          // one block had the whole unit and wrote it
        join_row<D>(p.part_o, p.part_ml, (int)(c1 - c0 + 1), [=](int c) { return (2ll * (c0 + c) + (c == 0)) * kDecodeRows + row; }, out);
    }
}

template <int D, int N>
cudaError_t launch_n(const DecodeParams& p, const SeqList<kMaxSeqs>& all, cudaStream_t stream) {
    SeqList<N> list;
    list.n = all.n;
    for (int i = 0; i < all.n; ++i) {
        list.row[i] = all.row[i];
        list.q_len[i] = all.q_len[i];
        list.seq[i] = all.seq[i];
    }
    const size_t smem = decode_smem(D, p.slots, all.n);
    const cudaError_t e = launch_chained(decode_kernel<D, N>, dim3(p.grid), kDecodeThreads, smem, stream, p, list);
    if (e != cudaSuccess) return e;
    const unsigned joins = (unsigned)std::min<long long>((long long)all.n * p.a.c.n_kv * p.most_rows, 8 * p.grid);
    return launch_chained(join_kernel<D, N>, dim3(joins), 128, 0, stream, p, list);
}

template <int D>
cudaError_t launch_d(const DecodeParams& p, const SeqList<kMaxSeqs>& l, cudaStream_t s) {
    return l.n <= kSmallSeqs ? launch_n<D, kSmallSeqs>(p, l, s) : launch_n<D, kMaxSeqs>(p, l, s);
}

template <int D>
cudaError_t opt_in() {
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, kSmallSeqs>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTwo);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(decode_kernel<D, kMaxSeqs>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTwo);
}

}  // namespace

size_t decode_smem(int dim, int slots, int seqs) {
    const size_t fixed = dim == 64 ? Layout<64>::kPrefix : dim == 128 ? Layout<128>::kPrefix : Layout<256>::kPrefix;
    return fixed + (size_t)(2 * seqs + 1) * 4 + 1024 + (size_t)slots * (dim == 64 ? kTile<64> : kTile<128>) * dim * 2;
}

cudaError_t decode_prepare_device() {
    cudaError_t e = opt_in<64>();
    if (e == cudaSuccess) e = opt_in<128>();
    if (e == cudaSuccess) e = opt_in<256>();
    return e;
}

cudaError_t launch_decode(const DecodeParams& p, const SeqList<kMaxSeqs>& seqs, cudaStream_t stream) {
    if (p.a.c.dim == 64) return launch_d<64>(p, seqs, stream);
    if (p.a.c.dim == 128) return launch_d<128>(p, seqs, stream);
    return launch_d<256>(p, seqs, stream);
}

}  // namespace lora
