// Attention of many new rows per sequence over the paged cache, on tcgen05.
//
// A unit is one key/value head and a run of its sequence's new rows: the rows of all query heads
// that share the head are packed into tiles of 128 (row r of a tile is query head r % g of token
// r / g), so that each tile of K and V is loaded once for all of them. Per cache tile of 128 tokens
//     S = Q K^T       tcgen05.mma, both operands in shared memory, 128 x 128 fp32 in tensor memory
//     P = 2^(S - m)   two threads per row: S to registers, P back to tensor memory in bf16 (the product
//                     takes bf16 operands; the sum l is of the unrounded fp32 weights)
//     O += P V        tcgen05.mma, P from tensor memory, V in shared memory as its rows lie there
// with the running maximum m and sum l of a softmax in base 2 per row. O is corrected only when a
// row's maximum grows by more than 2^8 (weights up to 2^8 keep bf16's relative precision; m, l and O
// always go by one reference), so a correction is rare after the first tile.
//
// The products are the bound (4 D flops a pair of row and token), and beside them what surrounds them:
// a product of N <= 128 costs its issuing warp ~90 cycles where the tensor cores need 64, and K and V
// land in shared memory at ~61 bytes a cycle. Heads of 64 and 128 run two tiles of rows per block in
// turn, so that one tile's products run while the other's weights are computed; a head of 256 (its O takes
// half of tensor memory) and calls of few rows have one tile and two score buffers. A block is persistent: softmax warps,
// an issuing warp or two, a TMA warp for K and V (one ring of pieces) that also hands out the work, and
// one for the queries and for blanking values that no row sees.
//
// Measured (one GB300, inputs past L2): a 4,096-row chunk at the end of 16,384 tokens 915 us with 24 / 12
// heads of 256 (1.58 PFLOP/s, 0.81 of the measured bf16 rate) and 1.13 to 1.16 ms with 48 / 8 heads of 128 (0.65);
// a 16,384-token prompt of 24 / 12 heads of 256, causal 2.01 ms (0.85), with a window of 4,096 1.00 ms (0.75);
// heads of 64 0.50 on a 4,096-row chunk.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_common.cuh"

namespace lora {
namespace {

using namespace dev;

constexpr int kTk = kPromptTile;

// Heads of D features; Q tiles of rows a block. (Heads of 64 and 128 have one where no sequence of the call needs
// two: drafts to verify, short chunks. Its next scores then run beside its weights, as in heads of 256, and the
// queries leave the ring more room: six chats with 8 draft rows over 60,000 tokens, 48 / 8 heads of 128 272 ->
// 256 us, of 64 235 -> 172; 64 prompts of 100 tokens, 16 heads of 64, 43 -> 35; none slower.)
template <int D, int Q>
struct Shape {
    static constexpr int kQ = Q;
    static constexpr int kS = Q == 1 ? 2 : 1;             // score buffers per tile
    static constexpr int kPieces = D == 256 ? 2 : 1;      // ring pieces of one tile of K (or of V)
    static constexpr int kPiece = D == 64 ? 16384 : 32768;
    static constexpr int kSlots = D == 256 ? 5 : D == 128 ? 7 - Q : Q == 2 ? 10 : 13;
    static constexpr int kQBytes = kTk * D * 2;
    static constexpr int kVTok = kTk / kPieces;           // tokens of one V piece
    static constexpr int kKChunks = D / 64 / kPieces;     // 64-feature chunks of one K piece
    static constexpr int kSoftmax = kQ * 256;             // softmax threads: two per row of a tile
    static constexpr bool kApart = D == 64 && Q == 2;               // weights beside the scores, not over them
    static constexpr int kIssuers = D == 64 && Q == 2 ? 2 : 1;      // warps that issue products
    static constexpr int kThreads = kSoftmax + kIssuers * 32 + 64;
    static constexpr int kO = 256;                        // first tensor-memory column of O (S: 128 each, from 0)
    static constexpr int kP = kApart ? 384 : 0;           // of the weights: 64 columns each, or in their scores' place
    static constexpr int kPStep = kApart ? 64 : 128;
    static constexpr int kRing = kQ * kQBytes;
    static constexpr int kBars = kRing + kSlots * kPiece;
    static constexpr int kPieceInfo = kBars + 512;        // [2] the pieces of work at hand
    static constexpr int kShare = kPieceInfo + 128;       // [kQ][128] floats between the two threads of a row
    static constexpr int kSmem = kShare + kQ * 512 + 1024;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32"
        " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
// Waits for the thread's loads from tensor memory; v, one of them, is used after the wait alone.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_wait16(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16],"
        " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operands are given by the low word of their descriptor (the address, and the leading
// offset); the high word is a constant: stride offset 1,024 bytes (8 rows of a 128-byte swizzle atom),
// version 1, 128-byte swizzle. The issuing warp shares its scheduler with softmax warps, so a
// product's operands cost one addition each.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t leading = 16) { return addr >> 4 | (leading >> 4) << 16; }

// D[tmem] (+)= A[smem] * B[smem]^T, bf16 operands with K contiguous.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint32_t pred) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(pred), "n"(kDescHi)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], A the bf16 weights as they lie in tensor memory. B is a tile of V as its
// rows lie in shared memory: features along N are contiguous (N-major), 64 of them per swizzled row; the
// descriptor's leading offset is the distance of its 64-feature chunks.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint32_t pred) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(pred), "n"(kDescHi)
        : "memory");
}

// A unit: one key/value head and a run of its sequence's new rows. Units go by sequence, then from the
// last rows (which see most) to the first, then by head.
struct Unit {
    int seq, head, tok0, q_len, row0, len;
    TileRange r;
};
template <int D, int Q, int N>
__device__ __forceinline__ Unit find_unit(const PromptParams& p, const PromptList<N>& list, int unit) {
    using S = Shape<D, Q>;
    Unit u;
    int lo = 0, hi = list.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list.unit0[mid] <= unit) lo = mid; else hi = mid - 1;
    }
    u.seq = list.seq[lo];
    u.q_len = list.q_len[lo];
    u.row0 = list.row[lo];
    const int step = S::kQ * p.tile_tokens, per = (u.q_len + step - 1) / step, v = unit - list.unit0[lo], n_kv = p.a.c.n_kv;
    u.head = v % n_kv;
    u.tok0 = (per - 1 - v / n_kv) * step;
    u.len = cache_len(p.a.c, u.seq);
    const int first = u.len - u.q_len + u.tok0, last = u.len - u.q_len + min(u.q_len, u.tok0 + step) - 1;
    u.r = tile_range(first, last, p.a.window, p.a.sinks, kTk);
    return u;
}

// The units are handed out one by one, those that see most first (a counter in global memory; which block
// has a unit does not change its output). Of the last ones, fewer than one a block, all tiles form one line
// that is cut into equal parts, one a block, where that saves more time than the join takes (kWorth tiles
// a block): a part may end inside a unit, whose sums then go to the workspace. Cut at any gain, or from 4 tiles on,
// 512 rows at the end of 2,048 tokens (48 / 8 heads of 128) take 86 us instead of 49, 8,192 causal rows of 16 heads
// of 128 279 instead of 248; never cut, six chats of 8 draft rows take 256 us instead of 72, a 4,096-row chunk at the
// end of 16,384 tokens 1,286 instead of 1,161. From 16 on gives what 8 gives in all of these.
constexpr int kWorth = 8;
struct Plan {
    uint32_t total;       // tiles of the last units, if they are cut (else 0)
    uint32_t blocks;      // blocks that get a part of them
};
__device__ __forceinline__ uint32_t part_begin(const Plan& l, uint32_t c) { return (uint32_t)((uint64_t)l.total * c / l.blocks); }
__device__ __forceinline__ uint32_t part_of(const Plan& l, uint32_t t) { return (uint32_t)(((uint64_t)(t + 1) * l.blocks - 1) / l.total); }
// From the last units' tiles and the longest of them.
__device__ __forceinline__ Plan plan_rest(const PromptParams& p, uint32_t total, uint32_t longest) {
    Plan l;
    const bool cut = (uint64_t)longest * p.blocks > total + (uint64_t)kWorth * p.blocks;
    l.total = cut ? total : 0;
    l.blocks = min((uint32_t)p.blocks, max(total, 1u));
    return l;
}
constexpr int kNoTile = -2;
// A piece of work as the producer hands it to the other warps, through shared memory.
struct Piece {
    int head, tok0, q_len, row0, len, s_tiles, lo_tile;     // its unit
    int t0, n;            // its tiles; n < 0: the end
    int part;             // where its sums go in the workspace; -1: to the output
    int two;              // its rows reach into the second tile
    int k0;               // its first piece in the ring's order
    // Its tiles with tokens that no row of the unit sees: gap and the one after it between the sinks and the window,
    // tail past the last token (kNoTile, or a tile outside [0, n): not in this piece).
    int gap, tail;
    int pad[2];
};
__device__ __forceinline__ bool at_edge(int gap, int tail, int t) { return (unsigned)(t - gap) < 2 || t == tail; }
static_assert(sizeof(Piece) == 64, "two pieces fill their place in shared memory");

// 32 bytes (a whole sector of L2) in one store; p is 32-byte aligned.
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// Two fp32 values in one instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    return (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

// Waits for several barriers at once: each lane brings one (and its parity). One shared-memory access
// of the warp then stands for all of them. Bounded like wait_bounded.
__device__ __forceinline__ bool wait_lanes(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, uint64_t limit_ns) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    bool mine = false;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            mine = mine || mbar_try_wait(bar, parity);
            if (__all_sync(0xffffffffu, mine)) return true;
        }
        const bool late = global_timer_ns() - t0 > limit_ns;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            if (late) {
                atomicOr(status, 1);
                *abort_flag = 1;
            }
            return false;
        }
    }
}
// The low n bits (n may be outside 0 .. 64).
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }
// The columns of 64 that a row sees: those up to hi that are lo or more, or below sk.
__device__ __forceinline__ uint64_t seen_bits(int hi, int lo, int sk) { return low_bits(hi + 1) & (~low_bits(lo) | low_bits(sk)); }
// Scores of 64 columns that the row does not see become -inf.
__device__ __forceinline__ void mask(uint32_t* v, uint64_t seen) {
    const uint32_t s0 = (uint32_t)seen, s1 = (uint32_t)(seen >> 32);
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        if (!(s0 & 1u << c)) v[c] = 0xff800000u;
        if (!(s1 & 1u << c)) v[32 + c] = 0xff800000u;
    }
}
template <int N>
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t* v) {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld32(taddr + c, v + c);
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld_wait32(v + c);
}
// Barrier of the two warps that share 32 rows; true for both if any thread of either wishes it.
__device__ __forceinline__ bool pair_any(int id, bool wish) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred p, %2, 64, q;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((int)wish), "r"(id)
        : "memory");
    return r != 0;
}
// The largest of three, and of N scores.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int N>
__device__ __forceinline__ float row_max(const uint32_t* v) {
    float x[8];                                            // eight chains
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = fmaxf(__uint_as_float(v[c]), __uint_as_float(v[8 + c]));
#pragma unroll
    for (int c = 16; c < N; c += 16)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = max3(x[e], __uint_as_float(v[c + e]), __uint_as_float(v[c + 8 + e]));
    return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
}
// N scores to weights 2^(s scl - ms): v[0 .. N / 2) get them in pairs, rounded to bf16 for the product with V;
// returns their sum before that rounding.
template <int N>
__device__ __forceinline__ float weights(uint32_t* v, float scl, float ms) {
    const uint64_t scl2 = pack2(scl, scl), ms2 = pack2(-ms, -ms);
    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
        const uint64_t e = fma2((uint64_t)v[2 * c + 1] << 32 | v[2 * c], scl2, ms2);
        const float x = ex2(lo2(e)), y = ex2(hi2(e));
        sum[c & 3] = add2(sum[c & 3], pack2(x, y));
        v[c] = pack_bf16x2(x, y);
    }
    sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
    return lo2(sum[0]) + hi2(sum[0]);
}

template <int D, int Q, int N>
__global__ void __launch_bounds__(Shape<D, Q>::kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ PromptList<N> list) {
    using S = Shape<D, Q>;
    extern __shared__ __align__(1024) uint8_t shared_bytes[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(shared_bytes) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + S::kBars);
    uint64_t* full = bars;                                // [kSlots] pieces of K and V
    uint64_t* empty = full + S::kSlots;
    uint64_t* raw = empty + S::kSlots;                    // [kSlots] pieces of V with tokens to blank, in their own order
    uint64_t* s_full = raw + S::kSlots;                   // [kQ * kS] scores
    uint64_t* p_full = s_full + 2;                        // [kQ * kS] weights (and O corrected)
    uint64_t* pv_done = p_full + 2;                       // [kQ * kS] product with V
    uint64_t* s_read = pv_done + 2;                       // [kQ] scores are in registers (kApart)
    uint64_t* q_full = s_read + 2;                        // [kQ] queries
    uint64_t* q_free = q_full + 2;                        // [kQ] their last scores are computed
    uint64_t* drain = q_free + 2;                         // [2] an issuer's last product
    uint64_t* turn = drain + 2;                           // [2] a tile's scores are issued
    uint64_t* told = turn + 2;                            // [2] a piece of work is there
    uint64_t* done = told + 2;                            // [2] and every warp has finished with it
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);              // known to be the same in every lane
    constexpr int kMmaWarp = S::kSoftmax / 32, kTmaWarp = kMmaWarp + S::kIssuers, kQueryWarp = kTmaWarp + 1;

    if (tid == 0) {
        for (int s = 0; s < S::kSlots; ++s) {
            mbar_init(smem_addr(&full[s]), 1);
            mbar_init(smem_addr(&empty[s]), S::kIssuers);   // every issuer that reads the piece
            mbar_init(smem_addr(&raw[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&s_full[s]), 1);
            mbar_init(smem_addr(&p_full[s]), 8);          // one arrival a warp
            mbar_init(smem_addr(&pv_done[s]), 1);
            mbar_init(smem_addr(&s_read[s]), 8);
            mbar_init(smem_addr(&q_full[s]), 1);
            mbar_init(smem_addr(&q_free[s]), 1);
            mbar_init(smem_addr(&drain[s]), 1);
            mbar_init(smem_addr(&turn[s]), 1);
            mbar_init(smem_addr(&told[s]), 1);
            mbar_init(smem_addr(&done[s]), S::kSoftmax / 32 + S::kIssuers + 1);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc<1>(smem_addr(tmem_slot), 512);
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    const AttnParams& a = p.a;
    const uint64_t limit = a.wait_limit_ns;
    griddep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Piece* const pieces = reinterpret_cast<Piece*>(base + S::kPieceInfo);
    griddep_launch_dependents();
    const uint32_t q_smem = smem_addr(base), ring = q_smem + S::kRing;
    const uint32_t issuer = lane == 0 ? 1u : 0u;
    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ producer
        const int gran = p.granule, per_tile = kTk / gran;
        const uint32_t box_bytes = (uint32_t)gran * 128;
        Unit u{};
        int t_end = 0;
        const int32_t* table = nullptr;
        // lane g < per_tile: the page and token of the tile's granule g; page -1: past the sequence
        auto place = [&](int t, int& page, int& tok) {
            page = -1;
            tok = 0;
            if (t >= t_end || lane >= per_tile) return;
            const int j = tile_token(u.r, t, kTk) + lane * gran;
            if (j >= u.len) return;
            const int pg = j / a.c.page_size;
            page = table[pg];
            tok = j - pg * a.c.page_size;
            if (page < 0 || page >= a.c.n_pages) page = a.c.n_pages;    // out of the map's range: zeros
        };
        // tiles until a stall that a test asks for (by units, not by pieces: a check in `load` cost a tenth of a
        // 4,096-row chunk's time with heads of 256)
        int allowed = a.debug_stall ? a.debug_stall - 1 : kNoStall;
        int slot = 0, issued = 0, edges = 0;                  // edges: pieces of V with tokens to blank
        uint32_t phase = 0, blanked = 0;                      // blanked: bit s, slot s holds one
        // Pieces of a tile of K (128 tokens x its share of the features) or of V (its share of the tokens x all). Those
        // of V at an edge are reported to the warp that blanks them, which reports them to the issuers.
        auto load = [&](bool v, int page, int tok, bool edge) -> bool {
#pragma unroll
            for (int x = 0; x < S::kPieces; ++x) {
                const int chunks = v ? D / 64 : S::kKChunks;
                const int grans = v ? S::kVTok / gran : per_tile;
                const int gi = lane / chunks, ch = lane - gi * chunks;
                const int from = (v ? x * grans : 0) + gi;
                const int pg = __shfl_sync(0xffffffffu, page, from & 31), tk = __shfl_sync(0xffffffffu, tok, from & 31);
                const bool mine = gi < grans && pg >= 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * box_bytes;
                if (!wait_warp(smem_addr(&empty[slot]), phase ^ 1, abort_flag, a.status, limit)) return false;
                const uint32_t bar = smem_addr(edge ? &raw[edges % S::kSlots] : &full[slot]);
                edges += edge;
                blanked = (blanked & ~(1u << slot)) | (uint32_t)edge << slot;
                mbar_arrive_expect_tx(bar, bytes, issuer);
                __syncwarp();
                if (mine)
                    tma_load_kv(ring + (uint32_t)slot * S::kPiece + (uint32_t)ch * ((v ? S::kVTok : kTk) * 128) + (uint32_t)gi * box_bytes,
                                v ? &p.tm_v : &p.tm_k, bar, v ? p.v_order : p.k_order,
                                ((v ? 0 : x * S::kKChunks) + ch) * 64, u.head, tk, pg);
                ++issued;
                if (++slot == S::kSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            return true;
        };
        // the last units' tiles: lane l has the sums before units l, l + 32, ... of them
        constexpr int kSums = (kPromptBlocks + 31) / 32;
        const int rest = p.units - p.whole;
        uint32_t before[kSums];
        Plan plan;
        {
            uint32_t carry = 0, longest = 0;
#pragma unroll
            for (int k = 0; k < kSums; ++k) {
                const int i = k * 32 + lane;
                before[k] = 0;
                if (k * 32 >= rest) continue;
                const uint32_t n = i < rest ? (uint32_t)find_unit<D, Q>(p, list, p.whole + i).r.n : 0;
                uint32_t v = n;
                longest = max(longest, n);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += x;
                }
                before[k] = carry + v - n;
                carry += __shfl_sync(0xffffffffu, v, 31);
                if (blockIdx.x == 0 && i < rest) p.prefix[i] = before[k];     // for the join
            }
            longest = __reduce_max_sync(0xffffffffu, longest);
            if (blockIdx.x == 0 && lane == 0) {
                p.prefix[rest] = carry;
                p.prefix[rest + 1] = longest;
            }
            plan = plan_rest(p, carry, longest);
        }
        const int whole = plan.total ? p.whole : p.units;     // units that are handed out
        uint32_t at = 0, end = 0;                             // this block's part of the others' tiles
        if (plan.total && blockIdx.x < plan.blocks) {
            at = part_begin(plan, blockIdx.x);
            end = part_begin(plan, blockIdx.x + 1);
        }
        bool ok = true;
        int count = 0;                                        // pieces so far
        int unit = (int)blockIdx.x;                           // the first ones go without the counter
        while (ok) {
            unit = __shfl_sync(0xffffffffu, unit, 0);
            int t0 = 0, t1 = 0, part = -1;
            const bool last = unit >= whole && at >= end;
            if (unit < whole) {
                u = find_unit<D, Q>(p, list, unit);
                t1 = u.r.n;
                if (lane == 0) unit = p.blocks + atomicAdd(p.counter, 1);     // the next one, while this one loads
            } else if (!last) {
                // the last unit that begins at or before the tile: not one without tiles
                int lo = -1;
                uint32_t from = 0;
#pragma unroll
                for (int k = 0; k < kSums; ++k) {
                    const uint32_t here = __ballot_sync(0xffffffffu, k * 32 + lane < rest && before[k] <= at);
                    const uint32_t x = __shfl_sync(0xffffffffu, before[k], here ? 31 - __clz(here) : 0);
                    if (here) {
                        lo = k * 32 + 31 - __clz(here);
                        from = x;
                    }
                }
                u = find_unit<D, Q>(p, list, p.whole + lo);
                t0 = (int)(at - from);
                t1 = (int)min((uint32_t)u.r.n, t0 + (end - at));
                if (t0 > 0 || t1 < u.r.n) part = 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
                at += (uint32_t)(t1 - t0);
            }
            ok = wait_warp(smem_addr(&done[count & 1]), (uint32_t)((count >> 1) & 1) ^ 1, abort_flag, a.status, limit);
            // After a wait that ran out nothing is written or told: a warp may still be at the piece in this place, and
            // where its rows go is read from it to the end. The abort flag ends the warps that listen.
            if (!ok) break;
            const int gap = a.window && u.r.first - a.window >= a.sinks ? u.r.s_tiles - 1 - t0 : kNoTile;
            const int tail = u.len % kTk ? u.r.s_tiles + u.len / kTk - u.r.lo_tile - t0 : kNoTile;
            if (lane == 0) {
                Piece& w = pieces[count & 1];
                w.head = u.head;
                w.tok0 = u.tok0;
                w.q_len = u.q_len;
                w.row0 = u.row0;
                w.len = u.len;
                w.s_tiles = u.r.s_tiles;
                w.lo_tile = u.r.lo_tile;
                w.t0 = t0;
                w.n = last ? -1 : t1 - t0;
                w.part = part;
                w.k0 = issued;
                w.gap = gap;
                w.tail = tail;
                w.two = S::kIssuers == 2 || u.q_len - u.tok0 > p.tile_tokens;
                mbar_arrive(smem_addr(&told[count & 1]));
            }
            __syncwarp();
            ++count;
            if (last) break;
            if (t0 == t1) continue;
            t_end = t1;
            table = a.c.table + u.seq * a.c.table_stride;
            const int t_stop = min(t1, t0 + allowed);
            if (a.debug_stall) allowed -= t_stop - t0;
            int page, tok, npage, ntok;
            place(t0, page, tok);
            place(t0 + 1, npage, ntok);
            ok = t0 < t_stop && load(false, page, tok, false);
            for (int t = t0; t < t_stop && ok; ++t) {
                int fpage, ftok;
                place(t + 2, fpage, ftok);
                const bool edge = at_edge(gap, tail, t - t0);
                if (S::kS == 2 || S::kApart) {
                    ok = (t + 1 == t1 || load(false, npage, ntok, false)) && load(true, page, tok, edge);
                } else {
                    ok = load(true, page, tok, edge) && (t + 1 == t1 || load(false, npage, ntok, false));
                }
                page = npage;
                tok = ntok;
                npage = fpage;
                ntok = ftok;
            }
            ok = ok && t_stop == t1;
        }
        // The copies in flight land before the block may end, whoever gave up.
        if (lane == 0) {
            for (int k = max(0, issued - S::kSlots); k < issued; ++k)
                if (!(blanked >> (k % S::kSlots) & 1))
                    wait_bounded(smem_addr(&full[k % S::kSlots]), (uint32_t)((k / S::kSlots) & 1), abort_flag, a.status, limit, false);
            for (int e = max(0, edges - S::kSlots); e < edges; ++e)
                wait_bounded(smem_addr(&raw[e % S::kSlots]), (uint32_t)((e / S::kSlots) & 1), abort_flag, a.status, limit, false);
            if (!ok) __threadfence();    // a unit may have been asked for and not waited for: before the counter is reset
        }
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------ queries, tokens to blank
        // Each piece's tiles of rows, as soon as the scores of the piece before are computed. (Loaded by the
        // softmax warps instead, a tile of 128 x 256 took 5 us: beside the ring the first cache level has
        // little room for loads in flight.) Then zeros in place of the values of tokens that no row of the unit
        // sees: they may hold anything, and their weight of 0 needs them finite. (By the softmax warps, before
        // their weights go out: 1,150 against 1,130 us for 4,096 rows of 128 at the end of 16,384 tokens and 185
        // against 175 for 16,384 rows of 128 with a window of 1,024; 985 against 994 with heads of 256 and a window
        // of 4,096, where this warp's hand-over is felt.)
        uint32_t used[2] = {0, 0};
        bool ok = true;
        int edges = 0;                                        // pieces of V blanked
        for (int count = 0; ok; ++count) {
            ok = wait_warp(smem_addr(&told[count & 1]), (uint32_t)(count >> 1) & 1, abort_flag, a.status, limit);
            if (!ok) break;
            const Piece& w = pieces[count & 1];
            const int n = w.n, head = w.head * p.group, two = w.two, row = w.row0 + w.tok0;
            const int gap = w.gap, tail = w.tail, k0 = w.k0, t0 = w.t0, s_tiles = w.s_tiles, lo_tile = w.lo_tile, len = w.len;
            const int lo = len - w.q_len + w.tok0 - a.window + 1;             // with a window: its first token
            __threadfence_block();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&done[count & 1]));
            if (n < 0) break;
            if (n == 0) continue;
#pragma unroll
            for (int q = 0; q < S::kQ; ++q) {
                if (q == 1 && !two) continue;
                ok = ok && wait_warp(smem_addr(&q_free[q]), (used[q] & 1) ^ 1, abort_flag, a.status, limit);
                if (!ok) break;
                const uint32_t bar = smem_addr(&q_full[q]);
                mbar_arrive_expect_tx(bar, (uint32_t)(p.tile_tokens * p.group) * D * 2, issuer);
                __syncwarp();
                const int token = row + q * p.tile_tokens;
                if (lane < D / 64)
                    tma_load_3d(q_smem + (uint32_t)(q * S::kQBytes + lane * (128 * 128)), &p.tm_q, bar, lane * 64, p.q_outer ? token : head,
                                p.q_outer ? head : token);
                ++used[q];
            }
            for (int i = 0; i < 3 && ok; ++i) {
                const int t = i < 2 ? gap + i : tail;
                if (t < 0 || t >= n || (i == 2 && t == gap + 1)) continue;
                const int at = t0 + t, from = (at < s_tiles ? at : lo_tile + at - s_tiles) * kTk;
                const int k = k0 + (S::kS == 2 || S::kApart ? S::kPieces * (2 * t + (t + 1 == n ? 1 : 2)) : 1 + 2 * t);   // V's pieces
#pragma unroll
                for (int x = 0; x < S::kPieces; ++x, ++edges) {
                    ok = ok && wait_warp(smem_addr(&raw[edges % S::kSlots]), (uint32_t)(edges / S::kSlots) & 1, abort_flag, a.status, limit);
                    if (!ok) break;
                    const uint32_t piece = ring + (uint32_t)((k + x) % S::kSlots) * S::kPiece;
                    const int tok = from + x * S::kVTok;
                    zero_tokens<D, S::kVTok>(piece, len - tok, S::kVTok, lane, 32);
                    if (a.window) zero_tokens<D, S::kVTok>(piece, a.sinks - tok, lo - tok, lane, 32);
                }
                if (!ok) break;
                fence_proxy_async_shared();
                __syncwarp();
                if (lane < S::kPieces) mbar_arrive(smem_addr(&full[(k + lane) % S::kSlots]));
            }
        }
        if (lane == 0)                   // as the producer's
            for (int q = 0; q < S::kQ; ++q)
                if (used[q]) wait_bounded(smem_addr(&q_full[q]), (used[q] - 1) & 1, abort_flag, a.status, limit, false);
    } else if (warp >= kMmaWarp) {
        // ------------------------------------------------------------ MMA issuers
        // A product of N = 128 or less costs the issuing warp ~90-105 cycles, more than the tensor cores need
        // for it (64 at N = 128), and a wait or an arrival holds the warp until the products it has issued are
        // done. So all that a tile needs is waited for at once, and its products then go back to back: those
        // with V, then the next scores. Two issuers, one per tile of rows, halve that cost but fall into step,
        // so that products and weights no longer overlap (4,096 rows at the end of 16,384 tokens, heads of
        // 128, at that step: 1,350 us with two, 1,297 with one). Heads of 64, where the weights bound the
        // tile, gain by two (8,192 causal: 221 against 240 us).
        const int me = warp - kMmaWarp;
        const uint32_t idesc_s = instr_desc_bf16(128, kTk);
        const uint32_t idesc_o = instr_desc_bf16(128, D) | 1u << 16;      // B is N-major
        bool ok = true;
        auto wait_on = [&](uint64_t* bar, uint32_t ph) { ok = ok && wait_warp(smem_addr(bar), ph & 1, abort_flag, a.status, limit); };
        // piece k of the ring's order
        auto wait_piece = [&](int k) { wait_on(&full[k % S::kSlots], (uint32_t)(k / S::kSlots)); };
        auto release = [&](int k) { mma_commit_local<1>(smem_addr(&empty[k % S::kSlots]), issuer); };
        // scores of tile q into buffer b from K piece k (the x-th of its tile)
        auto scores = [&](int q, int b, int k, int x) {
            const uint32_t kp = desc_lo(ring + (uint32_t)(k % S::kSlots) * S::kPiece);
            const uint32_t qp = desc_lo(q_smem + (uint32_t)q * S::kQBytes + (uint32_t)x * (S::kKChunks * 128 * 128));
#pragma unroll
            for (int c = 0; c < S::kKChunks; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_ss(tmem + (uint32_t)(q * S::kS + b) * 128, qp + ((c * (128 * 128) + j * 32) >> 4),
                           kp + ((c * (kTk * 128) + j * 32) >> 4), idesc_s, (x | c | j) != 0, issuer);
        };
        auto values = [&](int q, int b, int k, int x, bool add) {
            const uint32_t vp = desc_lo(ring + (uint32_t)(k % S::kSlots) * S::kPiece, S::kVTok * 128);
            const uint32_t wp = tmem + S::kP + (uint32_t)(q * S::kS + b) * S::kPStep + (uint32_t)x * (S::kVTok / 2);
#pragma unroll
            for (int j = 0; j < S::kVTok / 16; ++j)
                mma_ts(tmem + S::kO + (uint32_t)q * D, wp + j * 8, vp + (j * 2048 >> 4), idesc_o, add || (x | j) != 0, issuer);
        };
        // Tiles and units so far: the barriers' phases and the ring's pieces go by them.
        int tt = 0, units = 0, tt2 = 0, units2 = 0;               // the second tile has its own: it may be left out
        for (int count = 0; ok; ++count) {
            wait_on(&told[count & 1], (uint32_t)(count >> 1));
            if (!ok) break;
            const int n = pieces[count & 1].n, k0 = pieces[count & 1].k0;
            const bool two = pieces[count & 1].two;
            __threadfence_block();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&done[count & 1]));
            if (n < 0) break;
            if (n == 0) continue;
            if (S::kIssuers == 2) {
                // The ring's order: K(0), then per tile K(t + 1), V(t): the weights lie apart from the scores, so
                // the next scores need only the last ones read. The tiles of rows begin in turn, so that neither
                // runs ahead and holds the ring's pieces.
                wait_on(&q_full[me], (uint32_t)units);
                for (int t = -1; t < n && ok; ++t) {
                    const bool more = t + 1 < n;
                    if (more) {
                        const int next = tt + t + 1, k = k0 + (t < 0 ? 0 : 1 + 2 * t);
                        if (me == 1 || next > 0) wait_on(&turn[1 - me], (uint32_t)(me == 0 ? next - 1 : next));
                        if (next > 0) wait_on(&s_read[me], (uint32_t)(next - 1));
                        wait_piece(k);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive(smem_addr(&turn[me]));
                        tc_fence_after();
                        scores(me, 0, k, 0);
                        mma_commit_local<1>(smem_addr(&s_full[me]), issuer);
                        if (t + 2 == n) mma_commit_local<1>(smem_addr(&q_free[me]), issuer);
                        release(k);
                    }
                    if (t < 0) continue;
                    const int k = k0 + 1 + 2 * t + (more ? 1 : 0);
                    wait_on(&p_full[me], (uint32_t)(tt + t));
                    wait_piece(k);
                    if (!ok) break;
                    tc_fence_after();
                    values(me, 0, k, 0, t > 0);
                    mma_commit_local<1>(smem_addr(&pv_done[me]), issuer);
                    release(k);
                }
            } else if (S::kQ == 2) {
                // the ring's order: K(0), then per tile V(t), K(t + 1)
                for (int t = -1; t < n && ok; ++t) {
                    const int kv = k0 + 1 + 2 * t, ks = kv + 1;
#pragma unroll
                    for (int q = 0; q < S::kQ; ++q) {
                        if (q == 1 && !two) continue;
                        // lane 0 the weights (or the queries), and for both tiles at once 1 the piece of V, 2 that of K
                        uint64_t* bar = t >= 0 ? &p_full[q] : &q_full[q];
                        uint32_t ph = (uint32_t)(t >= 0 ? (q ? tt2 : tt) + t : q ? units2 : units);
                        if (q == 0 && t >= 0 && lane == 1) {
                            bar = &full[kv % S::kSlots];
                            ph = (uint32_t)(kv / S::kSlots);
                        }
                        if (q == 0 && t + 1 < n && lane == 2) {
                            bar = &full[ks % S::kSlots];
                            ph = (uint32_t)(ks / S::kSlots);
                        }
                        ok = ok && wait_lanes(smem_addr(bar), ph & 1, abort_flag, a.status, limit);
                        if (!ok) break;
                        tc_fence_after();
                        if (t >= 0) {
                            values(q, 0, kv, 0, t > 0);
                            mma_commit_local<1>(smem_addr(&pv_done[q]), issuer);
                        }
                        if (t + 1 < n) {
                            scores(q, 0, ks, 0);
                            mma_commit_local<1>(smem_addr(&s_full[q]), issuer);
                            if (t + 2 == n) mma_commit_local<1>(smem_addr(&q_free[q]), issuer);
                        }
                    }
                    if (!ok) break;
                    if (t >= 0) release(kv);
                    if (t + 1 < n) release(ks);
                }
            } else {
                // the ring's order: K(0), then per tile K(t + 1), V(t), one piece or two each
                for (int t = -1; t < n && ok; ++t) {
                    if (t + 1 < n) {
                        const int b = (tt + t + 1) & 1, k = k0 + (t < 0 ? 0 : S::kPieces * (2 * t + 1));
                        // lanes 0 and 1 a piece of K each, 2 the queries
                        const int kl = k + (lane & (S::kPieces - 1));
                        const bool first = t < 0 && lane == 2;
                        ok = wait_lanes(smem_addr(first ? q_full : &full[kl % S::kSlots]), (uint32_t)(first ? units : kl / S::kSlots) & 1,
                                        abort_flag, a.status, limit);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int x = 0; x < S::kPieces; ++x) {
                            scores(0, b, k + x, x);
                            release(k + x);
                        }
                        mma_commit_local<1>(smem_addr(&s_full[b]), issuer);
                        if (t + 2 == n) mma_commit_local<1>(smem_addr(&q_free[0]), issuer);
                    }
                    if (t < 0) continue;
                    const int b = (tt + t) & 1, k = k0 + S::kPieces * (2 * t + (t + 1 < n ? 2 : 1));
                    // lanes 0 and 1 a piece of V each, 2 the weights
                    const int kl = k + (lane & (S::kPieces - 1));
                    ok = wait_lanes(smem_addr(lane == 2 ? &p_full[b] : &full[kl % S::kSlots]),
                                    (uint32_t)(lane == 2 ? (tt + t) >> 1 : kl / S::kSlots) & 1, abort_flag, a.status, limit);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < S::kPieces; ++x) {
                        values(0, b, k + x, x, t > 0);
                        release(k + x);
                    }
                    mma_commit_local<1>(smem_addr(&pv_done[b]), issuer);
                }
            }
            tt += n;
            ++units;
            tt2 += two ? n : 0;
            units2 += two ? 1 : 0;
        }
        // every product has ended before tensor memory is given back
        mma_commit_local<1>(smem_addr(&drain[me]), issuer);
        if (lane == 0) wait_bounded(smem_addr(&drain[me]), 0, abort_flag, a.status, limit, false);
        __syncwarp();
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ softmax: two threads per row, 64 columns each
        const int q = warp >> 3, half = (warp >> 2) & 1, g = p.group;
        const int pair = 1 + q * 4 + (warp & 3);                         // named barrier of the two warps of these rows
        float* share = reinterpret_cast<float*>(base + S::kShare) + (q * 128 + (tid & 127));
        constexpr int kCols = kTk / 2, kOut = D / 2;                     // scores and features of this thread
        typedef __nv_bfloat16 bf;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);      // this warp's 32 lanes
        const uint32_t o_addr = lanes + S::kO + (uint32_t)q * D + (uint32_t)half * kOut;
        const float scl = a.scale_log2;
        // The piece at hand; what can be had from it again stays there, since a row's scores take most registers.
        int count = -1, n = 0, pos = -1;
        // This thread's row of the tile: its query head of the group, its token in the piece's sequence, and
        // whether there is one. (`row` is hidden from the compiler, which would keep the quotient otherwise.)
        auto row_of = [&](const Piece& u, int& tok, int& hg) {
            int row = tid & 127;
            asm volatile("" : "+r"(row));
            const int d = p.q_outer ? p.tile_tokens : g, x = row / d, y = row - x * d;
            const int qi = p.q_outer ? y : x;
            hg = p.q_outer ? x : y;
            tok = u.tok0 + q * p.tile_tokens + qi;
            return row < p.tile_tokens * g && tok < u.q_len;
        };
        auto out_row = [&](const Piece& u, int tok, int hg) {
            return static_cast<bf*>(a.out) + (long long)(u.row0 + tok) * a.o_stride + (u.head * g + hg) * a.o_head + half * kOut;
        };
        auto finish = [&](int c) {       // this warp needs piece c no more: what it has read of it is there
            __threadfence_block();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&done[c & 1]));
        };
        // The next piece: kReady, kNone where it has nothing for this tile of rows (the rows of a unit without
        // tiles are zeros), or kEnd. One piece at a time: the producer reuses a piece's place when every warp has
        // finished with the one before the last.
        enum { kReady, kNone, kEnd };
        auto advance = [&]() -> int {
            ++count;
            const bool there = wait_warp(smem_addr(&told[count & 1]), (uint32_t)(count >> 1) & 1, abort_flag, a.status, limit);
            if (pair_any(pair, !there)) return kEnd;             // the two warps of a row end together
            n = pieces[count & 1].n;
            if (n < 0) return kEnd;
            {
                const Piece& u = pieces[count & 1];
                int tok, hg;
                const bool valid = row_of(u, tok, hg);
                // a row without a token goes with the tile's last one, so that it asks for no mask of its own
                pos = u.len - u.q_len + min(min(tok, u.q_len - 1), u.tok0 + (q + 1) * p.tile_tokens - 1);
                if (n == 0 || (q == 1 && !u.two)) {
                    if (valid)
                        for (int c = 0; c < kOut / 8; ++c) reinterpret_cast<uint4*>(out_row(u, tok, hg))[c] = make_uint4(0, 0, 0, 0);
                    finish(count);
                    return kNone;
                }
            }
            return kReady;
        };
        int tt = 0;                      // tiles so far
        int state;
        while ((state = advance()) == kNone) {}
        while (state == kReady) {
        float m = -INFINITY, l = 0.f;
        // After a wait that ran out the warps run on without data, so that their barriers stay matched; the
        // status word says that the output is incomplete.
        for (int t = 0; t < n; ++t) {
            const int ti = tt + t, b = S::kS == 2 ? ti & 1 : 0;
            const uint32_t par = (uint32_t)(S::kS == 2 ? ti >> 1 : ti) & 1;
            const volatile Piece& u = pieces[count & 1];
            const int at_tile = u.t0 + t, s_tiles = u.s_tiles, j0 = (at_tile < s_tiles ? at_tile : u.lo_tile + at_tile - s_tiles) * kTk;
            wait_warp(smem_addr(&s_full[q * S::kS + b]), par, abort_flag, a.status, limit);
            tc_fence_after();
            const uint32_t s_addr = lanes + (uint32_t)(q * S::kS + b) * 128;
            const uint32_t p_addr = lanes + S::kP + (uint32_t)(q * S::kS + b) * S::kPStep + half * (kCols / 2);
            const int c0 = j0 + half * kCols;
            const int lo = a.window ? pos - a.window + 1 - c0 : 0, sk = a.window ? a.sinks - c0 : 0;
            const bool masked = __any_sync(0xffffffffu, pos - c0 < kCols - 1 || (lo > 0 && sk < kCols));
            // rows of which none sees a column here (past the diagonal, or before the window) have weights of zero
            const bool blind = masked && t > 0 && !__any_sync(0xffffffffu, seen_bits(pos - c0, lo, sk) != 0);
            uint32_t v[kCols];
            float top = -INFINITY, sum = 0.f;
            if (blind) {
#pragma unroll
                for (int c = 0; c < kCols / 2; ++c) v[c] = 0;
            } else {
                load_scores<kCols>(s_addr + half * kCols, v);
                if (masked) mask(v, seen_bits(pos - c0, lo, sk));
                top = row_max<kCols>(v);
            }
            // The weights by the reference at hand, while the row's other thread does its half; the barrier then
            // tells whether either maximum has outgrown the reference by 2^8 (or is the first), in which case both
            // read their scores again and go by a new one. It also orders the weights, which overwrite scores,
            // after both threads' reads. The first tile has no reference and goes the second way at once.
            const bool wish = m == -INFINITY ? top > -INFINITY : (top - m) * scl > 8.f;
            if (t > 0 && !blind) sum = weights<kCols>(v, scl, m == -INFINITY ? 0.f : m * scl);
            if (t == 0 || pair_any(pair, wish)) {
                if (half) *share = top;
                pair_any(pair, false);
                if (!half) *share = top = fmaxf(top, *share);
                pair_any(pair, false);
                if (half) top = *share;
                const bool grow = m == -INFINITY ? top > -INFINITY : (top - m) * scl > 8.f;
                const bool fix = grow && m != -INFINITY;
                if (__any_sync(0xffffffffu, fix)) {
                    const float alpha = fix ? ex2((m - top) * scl) : 1.f;
                    const int tp = ti - 1, bp = S::kS == 2 ? tp & 1 : 0;
                    wait_warp(smem_addr(&pv_done[q * S::kS + bp]), (S::kS == 2 ? tp >> 1 : tp) & 1, abort_flag, a.status, limit);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kOut / 16; ++c) {
                        uint32_t x[16];
                        tmem_ld16(o_addr + c * 16, x);
                        tmem_ld_wait16(x);
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
                        tmem_st16(o_addr + c * 16, x);
                    }
                    l *= alpha;
                }
                if (grow) m = top;
                if (t > 0) {
                    load_scores<kCols>(s_addr + half * kCols, v);
                    if (masked) mask(v, seen_bits(pos - c0, lo, sk));
                }
                sum = weights<kCols>(v, scl, m == -INFINITY ? 0.f : m * scl);
                if (t > 0) pair_any(pair, false);
            }
            if (S::kApart) {
                tc_fence_before();
                if (lane == 0) mbar_arrive(smem_addr(&s_read[q]));
                // the weights' place is free once the product before has ended
                if (t > 0) wait_warp(smem_addr(&pv_done[q]), (uint32_t)(ti - 1) & 1, abort_flag, a.status, limit);
                tc_fence_after();
            }
            l += sum;
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_st16(p_addr + c * 16, v + c * 16);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&p_full[q * S::kS + b]));
        }
        tt += n;
        // The next piece's scores are computed meanwhile. (Its first product with V waits for its weights, which
        // come after this thread has read O.)
        const int mine = count;
        {
            const int tp = tt - 1, bp = S::kS == 2 ? tp & 1 : 0;
            wait_warp(smem_addr(&pv_done[q * S::kS + bp]), (uint32_t)(S::kS == 2 ? tp >> 1 : tp) & 1, abort_flag, a.status, limit);
        }
        tc_fence_after();
        // the row's sum: its two threads' parts
        if (half) *share = l;
        pair_any(pair, false);
        if (!half) *share = l = l + *share;
        pair_any(pair, false);
        if (half) l = *share;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const Piece& u = pieces[mine & 1];
        int tok, hg;
        const int part = u.part;
        const bool store = row_of(u, tok, hg), to_out = part < 0;
        bf* const out = out_row(u, tok, hg);
        finish(mine);
        const long long at = ((long long)part * S::kQ + q) * 128 + (tid & 127);
        if (!to_out && half == 0) p.part_ml[at] = make_float2(m * scl, l);
#pragma unroll 1
        for (int c = 0; c < kOut / 32; ++c) {
            uint32_t x[32];
            tmem_ld32(o_addr + c * 32, x);
            tmem_ld_wait32(x);
            if (!store) continue;
            if (!to_out) {
                float* d = p.part_o + at * D + half * kOut + c * 32;
#pragma unroll
                for (int e = 0; e < 32; e += 8) store32(d + e, x + e);
            } else {
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    o[k] = pack_bf16x2(__uint_as_float(x[2 * k]) * inv, __uint_as_float(x[2 * k + 1]) * inv);
                if (p.out32) {
                    store32(out + c * 32, o);
                    store32(out + c * 32 + 16, o + 8);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4*>(out + c * 32 + e * 8) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
        }
        tc_fence_before();
        while ((state = advance()) == kNone) {}
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc<1>(tmem, 512);
    }
    // the last block to end leaves the counters as it found them
    if (tid == 0 && atomicAdd(p.counter + 1, 1) == p.blocks - 1) {
        p.counter[0] = 0;
        p.counter[1] = 0;
        __threadfence();
    }
}

// Joins the parts of the cut units, if they were cut: a block takes one row at a time. Also writes the
// zeros of cut units without a tile.
template <int D, int Q, int N>
__global__ void __launch_bounds__(128) prompt_join_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ PromptList<N> list) {
    using S = Shape<D, Q>;
    const int rest = p.units - p.whole, g = p.group, d = p.q_outer ? p.tile_tokens : g;
    griddep_wait();
    griddep_launch_dependents();
    const Plan plan = plan_rest(p, p.prefix[rest], p.prefix[rest + 1]);
    if (plan.total == 0) return;
    for (int i = blockIdx.x; i < rest * p.join_rows; i += gridDim.x) {
        const int unit = i / p.join_rows, row = i - unit * p.join_rows;
        const int q = row >> 7, r = row & 127, x = r / d, y = r - x * d, hg = p.q_outer ? x : y;
        const Unit u = find_unit<D, Q>(p, list, p.whole + unit);
        const int tok = u.tok0 + q * p.tile_tokens + (p.q_outer ? y : x);
        if (r >= p.tile_tokens * g || tok >= u.q_len) continue;
        const uint32_t first = p.prefix[unit], n = p.prefix[unit + 1] - first;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + (long long)(u.row0 + tok) * p.a.o_stride +
                             (u.head * g + hg) * p.a.o_head;
        if (n == 0) {
            for (int e = threadIdx.x; e < D; e += 128) out[e] = __float2bfloat16_rn(0.f);
            continue;
        }
        const uint32_t c0 = part_of(plan, first), c1 = part_of(plan, first + n - 1);
        if (c0 == c1) continue;          // one block had the whole unit and wrote it
        join_row<D>(p.part_o, p.part_ml, (int)(c1 - c0 + 1),
                    [=](int c) { return ((2ll * (c0 + c) + (c == 0)) * S::kQ + q) * 128 + r; }, out);
    }
}

template <int D, int Q, int N>
cudaError_t launch_n(const PromptParams& p, const PromptList<kMaxSeqs>& all, cudaStream_t stream) {
    PromptList<N> list;
    list.n = all.n;
    for (int i = 0; i < all.n; ++i) {
        list.row[i] = all.row[i];
        list.q_len[i] = all.q_len[i];
        list.seq[i] = all.seq[i];
        list.unit0[i] = all.unit0[i];
    }
    const cudaError_t e = launch_chained(prompt_kernel<D, Q, N>, dim3(p.blocks), Shape<D, Q>::kThreads, Shape<D, Q>::kSmem, stream, p, list);
    if (e != cudaSuccess || p.whole == p.units) return e;
    const unsigned joins = (unsigned)std::min((p.units - p.whole) * p.join_rows, 16 * p.blocks);
    return launch_chained(prompt_join_kernel<D, Q, N>, dim3(joins), 128, 0, stream, p, list);
}

template <int D, int Q>
cudaError_t launch_d(const PromptParams& p, const PromptList<kMaxSeqs>& l, cudaStream_t s) {
    return l.n <= kSmallSeqs ? launch_n<D, Q, kSmallSeqs>(p, l, s) : launch_n<D, Q, kMaxSeqs>(p, l, s);
}

template <int D, int Q>
cudaError_t opt_in() {
    cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D, Q, kSmallSeqs>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, Q>::kSmem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(prompt_kernel<D, Q, kMaxSeqs>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, Q>::kSmem);
}

}  // namespace

int prompt_tiles(int dim) { return dim == 256 ? 1 : 2; }

cudaError_t prompt_prepare_device() {
    cudaError_t e = opt_in<64, 1>();
    if (e == cudaSuccess) e = opt_in<64, 2>();
    if (e == cudaSuccess) e = opt_in<128, 1>();
    if (e == cudaSuccess) e = opt_in<128, 2>();
    if (e == cudaSuccess) e = opt_in<256, 1>();
    return e;
}

cudaError_t launch_prompt(const PromptParams& p, const PromptList<kMaxSeqs>& seqs, cudaStream_t stream) {
    if (p.a.c.dim == 64) return p.tiles == 1 ? launch_d<64, 1>(p, seqs, stream) : launch_d<64, 2>(p, seqs, stream);
    if (p.a.c.dim == 128) return p.tiles == 1 ? launch_d<128, 1>(p, seqs, stream) : launch_d<128, 2>(p, seqs, stream);
    return launch_d<256, 1>(p, seqs, stream);
}

}  // namespace lora
