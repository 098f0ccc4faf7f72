// sm_103a kernel of the projection with 8-bit activations and an 8-bit base weight:
//
//     acc[t, n]  = sum_g xs[t, g] ws[n / 128, g] sum_{k in group g} X[t, k] W[n, k]
//     acc[t, n] += U[t, :] B_a[n, :]^T        (adapter tiles; U from the bf16 shrink before this launch)
//     Y[t, n]    = bf16(acc[t, n])
//
// A group's 128 products are summed by tcgen05.mma kind::f8f6f4 in tensor memory; each group has a scale of
// its own per row and block of columns, so its sums leave tensor memory and are added, times that scale, to
// fp32 accumulators in the epilogue warps' registers. The expand is one more such block (kind::f16, bf16 operands, the
// stages of the whole rank where the ring is long enough) with scale 1, and one for each adapter of a tile that holds several.
//
// Per CTA: warp 0 loads the stages (TMA, rows of 128 bytes, 128-byte swizzle: 128 e4m3 or 64 bf16); warps 1 and
// 2 issue the even and the odd blocks' MMAs into the two TMEM buffers (a warp's barrier wait completes after the
// MMAs that it issued, so one warp's waits run under the other's MMAs); warp 3 owns TMEM and lays the blocks'
// scales out in shared memory; the others are the epilogue, two per TMEM lane quadrant, half of the columns each.
//
// What bounds it. Single CTAs: the fill of shared memory, 61 bytes a cycle (256 columns 48 KB a block, 0.42 us of the
// measured 0.46; 128 columns 0.28) or the weight's bytes. Pairs: a buffer's round trip, ~1,600 cycles from the issue of its
// MMAs over their end, the sums' reading and the release back to the issuer, of which four run at once: two buffers of
// two halves of 128 columns (9,728 rows of 5,120 -> 5,120 177 us, 0.43 us a block, 2.9 PFLOP/s; whole buffers of 256
// columns 197). Without the sums' reading 158.
//
// Every mbarrier wait is bounded by a wall-clock limit; a wait that runs out sets bit 0 of the status word and a
// CTA-wide abort flag, and all roles leave their loops, wait (bounded) for their own copies and MMAs in flight,
// free TMEM and return.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dev_common.cuh"
#include "lora_fp8.h"

namespace lora {
namespace dev {
namespace {

// D[tmem] (+)= A[smem] * B[smem]^T: e4m3 inputs (K = 32) or bf16 inputs (K = 16), fp32 accumulate; as mma_bf16.
template <int CG>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate, uint32_t pred) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(pred)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(pred)
            : "memory");
}
// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3 (format 0), both K-major, shape M x N.
__device__ __forceinline__ uint32_t instr_desc_e4m3(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tmem_wait16(uint32_t* v) {   // v, of the thread's loads, is used after the wait alone
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
// The warp's rows of Y in shared memory to global memory; the elected lane's group of copies.
__device__ __forceinline__ void store_rows(const CUtensorMap* map, uint32_t src, int col, int row) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Two fp32 values in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Arrive on another CTA's barrier without a release: what it orders is this warp's reads of tensor memory, which have
// completed (tcgen05.wait::ld, then the fence before it), and no write of this thread's. With the release, which waits
// for the thread's outstanding loads of scales, a block of the wide form took twice as long.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// One lane of a converged warp, the same one each time: commits are for the MMAs of the lane that issues them.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// wait_bounded and wait_warp of dev_common.cuh without the call: a kernel that deals its registers out anew makes none.
__device__ __forceinline__ bool wait_lane(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, uint64_t limit_ns,
                                          bool honour_abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (honour_abort && *abort_flag) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            atomicOr(status, 1);
            *abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, uint64_t limit_ns) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    int ok = 1;
    if ((threadIdx.x & 31) == 0) ok = wait_lane(bar, parity, abort_flag, status, limit_ns, true);
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The blocks of one unit as every role walks them: base groups [kb0, kb0 + nk), a stage each, then the expand's, of
// lora_stages stages; nb blocks and ns stages in all.
struct Work {
    Tile tile;
    int n0, kb0, nk, nb, ns;
    int e0;                                            // its first expand, where tiles hold several adapters
};
template <int CG, int NT, bool MERGED>
__device__ __forceinline__ Work decode(const Fp8Params& p, const Tile* tiles, int u, int rank, int part) {
    Work w;
    const int per = p.n_groups * p.raster_group;
    const int g = u / per, r = u - g * per;
    const int gw = min(p.raster_group, p.n_ntiles - g * p.raster_group);
    w.tile = tiles[(r / gw) * CG + rank];
    w.n0 = (g * p.raster_group + r % gw) * NT;
    w.kb0 = part * p.k_blocks / p.parts;
    w.nk = (part + 1) * p.k_blocks / p.parts - w.kb0;
    if (MERGED) {                                      // (the expands go to the parts of K in turn)
        const int e = part * w.tile.adapter / p.parts, mine = (part + 1) * w.tile.adapter / p.parts - e;
        w.e0 = w.tile.u_row + e;
        w.nb = w.nk + mine * p.expand_blocks;
        w.ns = w.nk + mine * p.k_lora;
        return w;
    }
    w.e0 = 0;
    const bool expand = w.tile.adapter && part == p.parts - 1;
    w.nb = w.nk + (expand ? p.expand_blocks : 0);
    w.ns = w.nk + (expand ? p.k_lora : 0);
    return w;
}

// In place of the scale of a row that takes nothing of an expand (a product's NaN is 0x7fffffff).
constexpr uint32_t kNothing = 0xffffffffu;

// The scales of a block, as warp 3 lays them out for the epilogue, and its unit's place.
struct ScaleSlot {
    float f[2][kTileM];                                // per half of the columns and row: xs ws, or kNothing
    int4 unit;                                         // first row, rows, first column (odd: kApart), blocks that its rows take
};

// CG: CTAs of the MMA's group; NT: columns of a TMEM buffer, half of them in each epilogue thread's registers. Registers
// of the launch are dealt out anew: the loading warps' to the accumulators (LOW x 128 + HIGH x 256 <= 384 x the launch's).
// MIXED: tiles hold several adapters (MERGED), or a pair's tiles differ in having one (APART). Forms of their own: the
// first in all of them cost the pairs a tenth, and more, the second 0.8 %.
template <int CG, int NT, int LOW, int HIGH, bool MIXED>
__global__ void __launch_bounds__(kFp8Threads, 1) lora_fp8_kernel(const __grid_constant__ Fp8Params p) {
    constexpr bool MERGED = MIXED && CG == 1, APART = MIXED && CG > 1;
    constexpr int EW = 8;                              // epilogue warps
    constexpr int kCols = NT / 2;                      // columns of an epilogue thread
    constexpr int kBufs = 512 / NT, kSlots = 2 * kBufs;   // TMEM buffers, places of scales
    constexpr int kHalves = CG, kHalf = NT / kHalves;  // a pair's columns in halves, each with its own MMAs and barriers:
                                                       // a warp of one half's sums waits for no other's (one issuing warp a half
                                                       // 195 us, both halves by the blocks' parity 177: file's head)
    constexpr int kYCols = CG > 1 ? 64 : 32;           // columns of a warp's part of the output at a time
    constexpr int kYStage = 64 * kYCols;               // its bytes
    static_assert(NT == 256 || (CG == 1 && NT == 128), "SM pairs run 256-column blocks");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int stages = p.stages;
    const uint32_t a_bytes = (uint32_t)p.a_rows * kFp8StageRow;
    const uint32_t b_bytes = (uint32_t)(NT / CG) * kFp8StageRow;
    // an A stage of fewer than 128 rows: the MMA's other rows read what follows in the rings, and are never stored
    uint8_t* a_ring = base;
    uint8_t* b_ring = a_ring + (size_t)stages * a_bytes;
    uint8_t* after = b_ring + (size_t)stages * b_bytes;
    uint8_t* y_stage = after;                          // the epilogue's output rows
    ScaleSlot* slots = reinterpret_cast<ScaleSlot*>(after + EW * kYStage);
    uint64_t* full = reinterpret_cast<uint64_t*>(slots + kSlots);
    uint64_t* empty = full + stages;
    uint64_t* tfull = empty + stages;
    uint64_t* tempty = tfull + kBufs * kHalves;
    uint64_t* drain = tempty + kBufs * kHalves;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // (uniform for the compiler too)
    const int cta = p.parts > 1 || CG > 1 ? (int)cluster_ctarank() : 0;
    const int rank = CG > 1 ? cta : 0, part = CG > 1 ? 0 : cta;
    const bool leader = rank == 0;
    const int span = CG * p.parts;                     // CTAs of a unit
    const int first = (int)blockIdx.x / span, step = (int)gridDim.x / span;
    const int n_units = p.n_groups * p.n_ntiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_addr(&full[s]), 1);
            mbar_init(smem_addr(&empty[s]), 1);
        }
        for (int b = 0; b < kBufs * kHalves; ++b) {          // (buffer by buffer)
            mbar_init(smem_addr(&tfull[b]), 2);              // the MMAs' commit, the scales
            mbar_init(smem_addr(&tempty[b]), CG * EW / kHalves);
        }
        mbar_init(smem_addr(drain), 2);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3) tmem_alloc<CG>(smem_addr(tmem_slot), 512);
    tc_fence_before();
    if (CG > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t limit = p.wait_limit_ns;
    const Tile* tiles = p.inline_wl ? p.inline_tiles : p.tiles;
    const CUtensorMap* bmaps = p.inline_wl ? p.inline_bmaps : p.tm_b;
    // Behind this call's own shrink, which began when the kernel before it had completed, the base runs beside the shrink:
    // only the warp that loads U waits for it (rank 256, 48 rows of 5,120 -> 12,288 25 -> 19 us, 2,048 rows of 6,144 -> 5,120
    // 93 -> 77, of 17,408 -> 5,120 220 -> 198). X, W and the scales are read without a wait of this grid's own: the kernel that
    // wrote them had completed, its writes performed, before the shrink began, but the model promises their visibility to the
    // grid that waits alone. It is so because they are read from L2, by TMA and past L1.
    if (!p.late_u) griddep_wait();
    griddep_launch_dependents();

    if (warp < 4) {
        regs_dec<LOW>();
        if (warp == 0 && !p.debug_stall) {
            // ------------------------------------------------------------ TMA producer
            int stage = 0, issued = 0, acquired = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t tx = CG * (a_bytes + b_bytes);
            for (int u = first; u < n_units && ok; u += step) {
                const Work w = decode<CG, NT, MERGED>(p, tiles, u, rank, part);
                const CUtensorMap* bm = &bmaps[w.ns > w.nk && !MERGED ? w.tile.adapter - 1 : 0];
                int u_row = w.tile.u_row, e = w.e0, ku = 0;
                if (w.ns > w.nk && !p.inline_wl && acquired != w.tile.adapter) {
                    tensormap_acquire(bm);
                    acquired = w.tile.adapter;
                }
                for (int b = 0; b < w.ns; ++b) {
                    if (!wait_all(smem_addr(&empty[stage]), phase ^ 1, abort_flag, p.status, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_addr(&full[stage]);
                    const uint32_t fb = CG > 1 ? map_to_rank(bar, 0) : bar;
                    const uint32_t sa = smem_addr(a_ring + (size_t)stage * a_bytes), sb = smem_addr(b_ring + (size_t)stage * b_bytes);
                    const bool main = b < w.nk;
                    const int k = main ? (w.kb0 + b) * kFp8Group : (MERGED ? ku : b - w.nk) * 64;
                    if (!main && p.late_u) griddep_wait();
                    if (MERGED && !main) {
                        if (ku == 0) {
                            bm = &bmaps[p.expand[e].adapter - 1];
                            u_row = p.expand[e++].slot * kTileM;
                        }
                        if (++ku == p.k_lora) ku = 0;
                    }
                    if (elect_one()) {
                        if (leader) mbar_arrive_expect_tx(bar, tx, 1u);
                        tma_load_2d<CG>(sa, main ? &p.tm_x : &p.tm_u, fb, k, main ? w.tile.row0 : MERGED ? u_row : w.tile.u_row, 1u);
                        if (CG == 1) {
                            tma_load_2d<CG>(sb, main ? &p.tm_w : bm, fb, k, w.n0, 1u);
                        } else {                             // a pair's CTA holds half of the columns of each half
                            tma_load_2d<CG>(sb, main ? &p.tm_w : bm, fb, k, w.n0 + rank * (kHalf / CG), 1u);
                            tma_load_2d<CG>(sb + kHalf / CG * kFp8StageRow, main ? &p.tm_w : bm, fb, k, w.n0 + kHalf + rank * (kHalf / CG), 1u);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                }
            }
            if (lane == 0) {
                const int from = issued > stages ? issued - stages : 0;
                // copies in flight (bounded, whatever the abort flag says); on SM pairs also the pair's last
                // releases of this CTA's stages: no remote arrive is pending when it exits
                if (!ok && leader)
                    for (int j = from; j < issued; ++j)
                        wait_lane(smem_addr(&full[j % stages]), (uint32_t)((j / stages) & 1), abort_flag, p.status, limit, false);
                if (CG > 1)
                    for (int j = from; j < issued; ++j)
                        wait_lane(smem_addr(&empty[j % stages]), (uint32_t)((j / stages) & 1), abort_flag, p.status, limit, false);
            }
        } else if ((warp == 1 || warp == 2) && leader) {
            // ------------------------------------------------------------ MMA issuers
            const uint32_t idesc8 = instr_desc_e4m3(kTileM * CG, kHalf), idesc16 = instr_desc_bf16(kTileM * CG, kHalf);
            constexpr uint64_t kHalfDesc = kHalf / CG * kFp8StageRow / 16;   // from one half's rows of B to the other's
            const int mine = warp - 1;                       // parity of the blocks this warp issues
            int stage = 0, blk = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = first; u < n_units && ok; u += step) {
                const Work w = decode<CG, NT, MERGED>(p, tiles, u, rank, part);
                for (int b = 0; b < w.nb; ++b, ++blk) {
                    const bool main = b < w.nk;
                    const int ns = main ? 1 : p.lora_stages;
                    if ((blk & 1) == mine) {
                        // The buffer first: it is free when the epilogue has taken block blk - kBufs, and so every stage up
                        // to that block's has been filled and read. Only then does a stage's parity tell this fill from the
                        // one a lap before, where a lap is no shorter than the stages of the blocks since (fp8_window).
                        const int buf = blk % kBufs;
                        const uint32_t d = tmem_base + (uint32_t)(buf * NT);
                        const uint32_t free = ((blk / kBufs) & 1) ^ 1;
                        ok = wait_all(smem_addr(&tempty[buf * kHalves]), free, abort_flag, p.status, limit);
                        for (int s = 0; s < ns && ok; ++s) {
                            ok = wait_all(smem_addr(&full[stage]), phase, abort_flag, p.status, limit);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t ad = smem_desc<64>(smem_addr(a_ring + (size_t)stage * a_bytes));
                            const uint64_t bd = smem_desc<64>(smem_addr(b_ring + (size_t)stage * b_bytes));
#pragma unroll
                            for (int h = 0; h < kHalves; ++h) {
                                if (h > 0 && s == 0) {
                                    ok = wait_all(smem_addr(&tempty[buf * kHalves + h]), free, abort_flag, p.status, limit);
                                    if (!ok) break;
                                    tc_fence_after();
                                }
                                // 32 bytes along K inside the swizzled rows a step
                                // (one elected lane, in a branch of its own: 4 MMAs issue in ~100 cycles; under a predicate
                                // that the compiler cannot tell to be one lane's, in ~550)
                                if (elect_one()) {
                                    const uint64_t hd = bd + h * kHalfDesc;
                                    if (main) {
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            mma_e4m3<CG>(d + h * kHalf, ad + (uint64_t)(2 * k), hd + (uint64_t)(2 * k), idesc8, k > 0 ? 1u : 0u, 1u);
                                    } else {
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            mma_bf16<CG>(d + h * kHalf, ad + (uint64_t)(2 * k), hd + (uint64_t)(2 * k), idesc16, (s > 0 || k > 0) ? 1u : 0u, 1u);
                                    }
                                    if (s == ns - 1) mma_commit<CG>(smem_addr(&tfull[buf * kHalves + h]), 1u);
                                    if (h == kHalves - 1) mma_commit<CG>(smem_addr(&empty[stage]), 1u);
                                }
                                __syncwarp();
                            }
                            if (!ok) break;
                            if (++stage == stages) { stage = 0; phase ^= 1; }
                        }
                        if (!ok) break;
                    } else {
                        stage += ns;
                        if (stage >= stages) { stage -= stages; phase ^= 1; }
                    }
                }
            }
            // every MMA this warp issued has completed before TMEM is released
            if (elect_one()) mma_commit_local<CG>(smem_addr(drain), 1u);
            __syncwarp();
            if (lane == 0) wait_lane(smem_addr(drain), 0, abort_flag, p.status, limit, false);
        }
        if (warp == 3) {
            // ------------------------------------------------------------ scales, kBufs blocks ahead
            const int G = p.k_blocks;
            int blk = 0;
            bool ok = true;
            for (int u = first; u < n_units && ok; u += step) {
                const Work w = decode<CG, NT, MERGED>(p, tiles, u, rank, part);
                // (rows and columns past the unit's last take that one's; read from L2, as TMA reads: nothing of an earlier launch's
                // L1 is used where this one did not wait)
                const float *xs[4], *ws[2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    xs[i] = p.xs + (long long)min(w.tile.row0 + min(lane + 32 * i, max(w.tile.nrows - 1, 0)), p.rows - 1) * G;
#pragma unroll
                for (int h = 0; h < 2; ++h) ws[h] = p.ws + (long long)(min(w.n0 + h * kCols, p.d_out - 1) >> 7) * G;
                for (int b0 = 0; b0 < w.nb && ok; b0 += 4) {
                    const int g = w.kb0 + b0;
                    auto take = [&](const float* s, float* v) {   // (past the last group: never used)
                        if (p.vec_scales && (g & 3) == 0 && g < G) {
                            *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(s + g));
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) v[k] = __ldcg(s + min(g + k, G - 1));
                        }
                    };
                    float c[2][4], x[4][4];                  // four blocks' loads in flight
                    take(ws[0], c[0]);
                    take(ws[1], c[1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) take(xs[i], x[i]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (b0 + k >= w.nb) break;
                        // Block blk - kBufs's sums are there: its MMAs began when the epilogue had read block blk - 2 kBufs,
                        // its scales with it. And blk's phase of the barrier has begun.
                        const int buf = blk % kBufs;
#pragma unroll
                        for (int h = 0; h < kHalves && ok; ++h)
                            if (blk >= kBufs) ok = wait_all(smem_addr(&tfull[buf * kHalves + h]), (blk / kBufs - 1) & 1, abort_flag, p.status, limit);
                        if (!ok) break;
                        ScaleSlot& slot = slots[blk % kSlots];
                        if (MERGED && b0 + k >= w.nk) {
                            const uint32_t* rows = p.expand[w.e0 + (b0 + k - w.nk) / p.expand_blocks].rows;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                slot.f[0][lane + 32 * i] = slot.f[1][lane + 32 * i] = rows[i] >> lane & 1 ? 1.f : __uint_as_float(kNothing);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int h = 0; h < 2; ++h) slot.f[h][lane + 32 * i] = b0 + k < w.nk ? x[i][k] * c[h][k] : 1.f;
                        }
                        const bool apart = APART && w.tile.split_index == kApart;
                        if (lane == 0) slot.unit = make_int4(w.tile.row0, w.tile.nrows, w.n0 | (int)apart, apart ? w.nk : w.nb);
                        __syncwarp();
                        if (lane < kHalves) mbar_arrive(smem_addr(&tfull[buf * kHalves + lane]));
                        ++blk;
                    }
                }
            }
        }
        __syncwarp();
        if (p.late_u && warp == 0) griddep_wait();           // (this launch does not end before the shrink, whatever it met)
        if (CG == 1 && p.parts > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        // ------------------------------------------------------------ epilogue
        regs_inc<HIGH>();
        const int q = warp & 3, cg = (warp - 4) >> 2;        // TMEM lane quadrant, group of columns
        const int r_local = q * 32 + lane;
        const uint32_t t0 = tmem_base + (uint32_t)(cg * kCols) + ((uint32_t)(q * 32) << 16);
        uint8_t* const mine = y_stage + (warp - 4) * kYStage;
        const uint32_t my_scale = smem_addr(&slots[0].f[cg][r_local]);
        const int half = kHalves > 1 ? cg : 0;               // of the block's columns: this warp's barriers
        const uint32_t tfull0 = smem_addr(tfull + half);
        const uint32_t tempty0 = CG > 1 ? map_to_rank(smem_addr(tempty + half), 0) : smem_addr(tempty + half);
        uint32_t buf = 0, phase = 0, place = 0;
        bool ok = true;
        uint64_t acc[kCols / 2];
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
        for (int u = first; u < n_units && ok; u += step) {
            int row0 = 0, nrows = 0, n0 = 0, nb = 1;
#pragma unroll 1
            for (int b = 0; b < nb; ++b) {
                if (!wait_all(tfull0 + 8 * kHalves * buf, phase, abort_flag, p.status, limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                {
                    float f;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(my_scale + place * (uint32_t)sizeof(ScaleSlot)));
                    if (b == 0) {
                        const int4 unit = slots[place].unit;
                        row0 = unit.x;
                        nrows = unit.y;
                        n0 = unit.z;
                        nb = unit.w;
                    }
                    const uint32_t t = t0 + buf * NT;
                    const uint64_t f2 = pair(__float_as_uint(f), __float_as_uint(f));
                    auto release = [&] {                     // this warp has read the buffer
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (CG > 1) arrive_relaxed(tempty0 + 8 * kHalves * buf);
                            else mbar_arrive(tempty0 + 8 * kHalves * buf);
                        }
                    };
                    if (CG == 1 && q * 32 >= nrows) {        // no row of the unit's lies here
                        release();
                    } else if (MERGED && __any_sync(0xffffffffu, __float_as_uint(f) == kNothing)) {
                        uint32_t v[16];
#pragma unroll
                        for (int c = 0; c < kCols / 16; ++c) {
                            tmem_ld16(t + 16 * c, v);
                            tmem_wait16(v);
                            if (c + 1 == kCols / 16) release();
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (__float_as_uint(f) != kNothing) acc[8 * c + i] = fma2(pair(v[2 * i], v[2 * i + 1]), f2, acc[8 * c + i]);
                        }
                    } else {                                 // the next columns' load runs under these ones' sums
                        uint32_t v[2][16];
                        tmem_ld16(t, v[0]);
#pragma unroll
                        for (int c = 0; c < kCols / 16; ++c) {
                            tmem_wait16(v[c & 1]);
                            if (c + 1 < kCols / 16) tmem_ld16(t + 16 * (c + 1), v[(c + 1) & 1]);
                            else release();
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                acc[8 * c + i] = fma2(pair(v[c & 1][2 * i], v[c & 1][2 * i + 1]), f2, acc[8 * c + i]);
                        }
                    }
                    if (++buf == kBufs) { buf = 0; phase ^= 1; }
                    place = place + 1 == kSlots ? 0 : place + 1;
                }
            }
            if (APART && (n0 & 1)) {                         // the partner's expand, unread
                n0 &= ~1;
#pragma unroll 1
                for (int b = 0; b < p.expand_blocks && ok; ++b) {
                    ok = wait_all(tfull0 + 8 * kHalves * buf, phase, abort_flag, p.status, limit);
                    if (!ok) break;
                    if (lane == 0) arrive_relaxed(tempty0 + 8 * kHalves * buf);
                    if (++buf == kBufs) { buf = 0; phase ^= 1; }
                    place = place + 1 == kSlots ? 0 : place + 1;
                }
            }
            if (!ok) break;
            if (CG > 1 || p.parts == 1) {
                // The thread's row goes through the warp's part of shared memory, kYCols columns of 32 rows at a time, its 16-byte
                // pieces swizzled by row as a tensor map's. A tile whose last row is its 128th or the batch's last leaves it
                // as TMA copies (clipped at the batch's end); another one's rows are followed by the next tile's, and kYCols / 8
                // lanes write a row together. (Rows stored by their threads, 16 bytes here and there, took 9,400 cycles a
                // 256 x 256 unit, lanes together 2,600.)
                constexpr int kPieces = kYCols / 8, kShift = kPieces == 4 ? 1 : 0;
                const bool copy = (nrows == kTileM || row0 + nrows == p.rows) && q * 32 < nrows;
#pragma unroll
                for (int h = 0; h < kCols / kYCols; ++h) {
                    if (lane == 0) stores_read();            // (the group before has left the buffer)
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        {
                            uint64_t* a = acc + kYCols / 2 * h + 4 * c;
                            *reinterpret_cast<uint4*>(mine + lane * kYCols * 2 + ((c ^ ((lane >> kShift) & (kPieces - 1))) << 4)) =
                                make_uint4(pack_bf16x2(lo2(a[0]), hi2(a[0])), pack_bf16x2(lo2(a[1]), hi2(a[1])),
                                           pack_bf16x2(lo2(a[2]), hi2(a[2])), pack_bf16x2(lo2(a[3]), hi2(a[3])));
                            a[0] = a[1] = a[2] = a[3] = 0;
                        }
                    }
                    const int first_col = n0 + cg * kCols + kYCols * h;
                    if (copy) {
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0 && first_col < p.d_out) store_rows(&p.tm_y, smem_addr(mine), first_col, row0 + q * 32);
                        continue;
                    }
                    __syncwarp();
                    const int c = lane & (kPieces - 1), col = first_col + 8 * c;
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.y) + (long long)(row0 + q * 32) * p.d_out + col;
                    const int n = col < p.d_out ? nrows - q * 32 : 0;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int r = 32 / kPieces * i + lane / kPieces;
                        if (r < n)
                            *reinterpret_cast<uint4*>(out + (long long)r * p.d_out) =
                                *reinterpret_cast<const uint4*>(mine + r * kYCols * 2 + ((c ^ ((r >> kShift) & (kPieces - 1))) << 4));
                    }
                }
            } else {
                // every stage has been read (the MMAs' commits): this part's sums take the rings' place, four
                // columns of the 128 rows side by side
                float4* sums = reinterpret_cast<float4*>(base);
#pragma unroll
                for (int c = 0; c < kCols / 4; ++c)
                    if (q * 32 < nrows)
                        sums[(cg * (kCols >> 2) + c) * 128 + r_local] =
                            make_float4(lo2(acc[2 * c]), hi2(acc[2 * c]), lo2(acc[2 * c + 1]), hi2(acc[2 * c + 1]));
            }
        }
        if (lane == 0) stores_read();                        // before the CTA's shared memory goes
        if (CG == 1 && p.parts > 1) {
            __syncwarp();
            cluster_sync();
            if (ok) {
                // each CTA adds its share of the columns over the parts, in their order
                const Work w = decode<CG, NT, MERGED>(p, tiles, first, rank, part);
                const int v0 = part * (NT / 8) / p.parts, vecs = (part + 1) * (NT / 8) / p.parts - v0;
                for (int i = (int)threadIdx.x - 128; i < w.tile.nrows * vecs; i += 32 * EW) {
                    const int r = i / vecs, c = 8 * (v0 + i - r * vecs);
                    if (w.n0 + c >= p.d_out) continue;
                    const uint32_t at = smem_addr(base) + (uint32_t)(((c >> 2) * 128 + r) * 16);
                    float s[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[k] = 0.f;
                    for (int j0 = 0; j0 < p.parts; j0 += 2) {   // two parts' loads in flight
                        const int j1 = min(j0 + 1, p.parts - 1);
                        const uint32_t a0 = map_to_rank(at, (uint32_t)j0), a1 = map_to_rank(at, (uint32_t)j1);
                        const float4 x0 = ld_cluster(a0), y0 = ld_cluster(a0 + 128 * 16), x1 = ld_cluster(a1), y1 = ld_cluster(a1 + 128 * 16);
                        s[0] += x0.x; s[1] += x0.y; s[2] += x0.z; s[3] += x0.w;
                        s[4] += y0.x; s[5] += y0.y; s[6] += y0.z; s[7] += y0.w;
                        if (j1 > j0) {
                            s[0] += x1.x; s[1] += x1.y; s[2] += x1.z; s[3] += x1.w;
                            s[4] += y1.x; s[5] += y1.y; s[6] += y1.z; s[7] += y1.w;
                        }
                    }
                    uint4 o;
                    o.x = pack_bf16x2(s[0], s[1]);
                    o.y = pack_bf16x2(s[2], s[3]);
                    o.z = pack_bf16x2(s[4], s[5]);
                    o.w = pack_bf16x2(s[6], s[7]);
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + (long long)(w.tile.row0 + r) * p.d_out + w.n0 + c) = o;
                }
            }
            __syncwarp();
            cluster_sync();                                  // the parts' sums have been read
        }
    }
    __syncwarp();
    tc_fence_before();
    if (CG > 1) cluster_sync();                              // neither CTA of the pair touches the other's memory after this
    else __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, 512);
    }
}

// U[t, :] = bf16(s_a X[t, :] A_a^T) for one tile of 128 rows, n columns of the rank and one part of K a unit, the parts of a
// tile a cluster; a CTA takes one unit after another where there are more than CTAs, its K whole then. The bf16 kernel's shrink units take a tile's whole K each, 272 K steps of it at d_in 17,408 (1,553 rows
// of rank 64 there 80 us; in 8 parts 12). Bound by the fill of shared memory, 61 bytes a cycle and SM.
__global__ void __launch_bounds__(kShrinkThreads, 1) lora_shrink_kernel(const __grid_constant__ ShrinkParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int stages = p.stages;
    const uint32_t a_bytes = kTileM * kFp8StageRow, b_bytes = (uint32_t)p.n * kFp8StageRow;
    uint8_t* a_ring = base;
    uint8_t* b_ring = a_ring + (size_t)stages * a_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(b_ring + (size_t)stages * b_bytes);
    uint64_t* empty = full + stages;
    uint64_t* done = empty + stages;                   // a unit's MMAs have completed
    uint64_t* taken = done + 1;                        // and its sums have been read
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(taken + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int part = p.parts > 1 ? (int)cluster_ctarank() : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_addr(&full[s]), 1);
            mbar_init(smem_addr(&empty[s]), 1);
        }
        mbar_init(smem_addr(done), 1);
        mbar_init(smem_addr(taken), 4);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<1>(smem_addr(tmem_slot), 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t limit = p.wait_limit_ns;
    griddep_wait();
    griddep_launch_dependents();

    const int n_units = p.n_tiles * p.rank_tiles, first = (int)blockIdx.x / p.parts, step = (int)gridDim.x / p.parts;
    const int k0 = part * p.k_steps / p.parts, nk = (part + 1) * p.k_steps / p.parts - k0;
    Tile tile;                                         // of a unit, and its columns of the rank
    int c0, cols;
    auto place = [&](int unit) {
        tile = (p.inline_wl ? p.inline_tiles : p.tiles)[unit / p.rank_tiles];
        c0 = unit % p.rank_tiles * p.n;
        cols = min(p.n, p.rank - c0);
    };
    place(first);
    bool ok = true;
    if (warp == 0 && !p.debug_stall) {
        int issued = 0, stage = 0;
        uint32_t phase = 0;
        for (int unit = first; unit < n_units && ok; unit += step) {
            if (unit != first) place(unit);
            const CUtensorMap* am = &(p.inline_wl ? p.inline_amaps : p.tm_a)[tile.adapter - 1];
            if (!p.inline_wl) tensormap_acquire(am);
            for (int k = 0; k < nk; ++k) {
                if (!wait_all(smem_addr(&empty[stage]), phase ^ 1, abort_flag, p.status, limit)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_addr(&full[stage]);
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, a_bytes + b_bytes, 1u);
                    tma_load_2d<1>(smem_addr(a_ring + (size_t)stage * a_bytes), &p.tm_x, bar, (k0 + k) * 64, tile.row0, 1u);
                    tma_load_2d<1>(smem_addr(b_ring + (size_t)stage * b_bytes), am, bar, (k0 + k) * 64, c0, 1u);
                }
                __syncwarp();
                ++issued;
                if (++stage == stages) { stage = 0; phase ^= 1; }
            }
        }
        if (!ok && lane == 0)                              // copies in flight (bounded, whatever the abort flag says)
            for (int j = issued > stages ? issued - stages : 0; j < issued; ++j)
                wait_lane(smem_addr(&full[j % stages]), (uint32_t)((j / stages) & 1), abort_flag, p.status, limit, false);
    } else if (warp == 1) {
        const uint32_t idesc = instr_desc_bf16(kTileM, p.n);
        int stage = 0, n = 0;                              // n: units before this one
        uint32_t phase = 0;
        for (int unit = first;; unit += step, ++n) {
            if (n > 0) {                                   // the unit before has been read
                ok = wait_all(smem_addr(taken), (n - 1) & 1, abort_flag, p.status, limit);
                tc_fence_after();
            }
            for (int k = 0; k < nk && ok; ++k) {
                ok = wait_all(smem_addr(&full[stage]), phase, abort_flag, p.status, limit);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ad = smem_desc<64>(smem_addr(a_ring + (size_t)stage * a_bytes));
                const uint64_t bd = smem_desc<64>(smem_addr(b_ring + (size_t)stage * b_bytes));
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_bf16<1>(tmem_base, ad + (uint64_t)(2 * i), bd + (uint64_t)(2 * i), idesc, (k > 0 || i > 0) ? 1u : 0u, 1u);
                    mma_commit<1>(smem_addr(&empty[stage]), 1u);
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; phase ^= 1; }
            }
            // (also where a wait ran out: every MMA this warp issued completes before TMEM is released)
            if (elect_one()) mma_commit<1>(smem_addr(done), 1u);
            __syncwarp();
            if (!ok || unit + step >= n_units) break;
        }
        if (lane == 0) wait_lane(smem_addr(done), n & 1, abort_flag, p.status, limit, false);
    }
    __syncwarp();
    float4* sums = reinterpret_cast<float4*>(base);
    for (int unit = first, n = 0; warp >= 4 && unit < n_units; unit += step, ++n) {
        // ------------------------------------------------------------ epilogue: row 32 q + lane
        if (unit != first) place(unit);
        const int q = warp & 3, r_local = q * 32 + lane, row = tile.row0 + r_local;
        ok = wait_all(smem_addr(done), n & 1, abort_flag, p.status, limit) && !*abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (q * 32 < tile.nrows) {
            const bool mine = r_local < tile.nrows;
            const int32_t* seg_off = p.inline_wl ? p.inline_seg : p.seg_off;
            const int32_t* seg_id = p.inline_wl ? p.inline_seg + p.n_seg + 1 : p.seg_id;
            const float s = mine && row_adapter(seg_off, seg_id, p.n_seg, row) == tile.adapter
                                ? (p.inline_wl ? p.inline_scales : p.scales)[tile.adapter - 1] : 0.f;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.u) + (long long)(tile.u_row + r_local) * p.rank + c0;
            for (int c = 0; c < p.n; c += 16) {
                uint32_t v[16];
                if (nk) tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)c, v);
                tmem_wait16(v);
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = nk && s != 0.f ? __uint_as_float(v[i]) * s : 0.f;
                if (p.parts > 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sums[((c >> 2) + i) * kTileM + r_local] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                } else if (mine) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (c + 8 * i < cols)
                            *reinterpret_cast<uint4*>(out + c + 8 * i) =
                                make_uint4(pack_bf16x2(f[8 * i], f[8 * i + 1]), pack_bf16x2(f[8 * i + 2], f[8 * i + 3]),
                                           pack_bf16x2(f[8 * i + 4], f[8 * i + 5]), pack_bf16x2(f[8 * i + 6], f[8 * i + 7]));
                }
            }
        }
        if (unit + step >= n_units) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(taken));
    }
    if (p.parts > 1) {                                     // (one unit a cluster)
        __syncwarp();
        cluster_sync();
        if (warp >= 4 && ok) {
            // each CTA adds its share of the columns over the parts, in their order
            const int v0 = part * (cols / 8) / p.parts, vecs = (part + 1) * (cols / 8) / p.parts - v0;
            for (int i = (int)threadIdx.x - 128; i < tile.nrows * vecs; i += 128) {
                const int r = i / vecs, c = 8 * (v0 + i - r * vecs);
                const uint32_t at = smem_addr(base) + (uint32_t)(((c >> 2) * kTileM + r) * 16);
                float s[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] = 0.f;
                for (int j = 0; j < p.parts; ++j) {
                    const uint32_t a = map_to_rank(at, (uint32_t)j);
                    const float4 x = ld_cluster(a), y = ld_cluster(a + kTileM * 16);
                    s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
                    s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
                }
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.u) + (long long)(tile.u_row + r) * p.rank + c0 + c) =
                    make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
            }
        }
        __syncwarp();
        cluster_sync();                                    // the parts' sums have been read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, 256);
    }
}

}  // namespace
}  // namespace dev

namespace {
// 384 threads of 168 registers, dealt out anew: 72 x 128 + 216 x 256 = 168 x 384. A few bytes spilled in the loading warps
// cost a tenth to a fifth of all (pairs with buffers of 256 columns, 9,728 rows of 5,120 -> 5,120: 198 us; with 64 and 216,
// 40 bytes, 223).
constexpr auto kWide = dev::lora_fp8_kernel<2, 256, 72, 216, false>, kWideApart = dev::lora_fp8_kernel<2, 256, 72, 216, true>;
constexpr auto kSingle = dev::lora_fp8_kernel<1, 256, 72, 216, false>, kSingleMerged = dev::lora_fp8_kernel<1, 256, 72, 216, true>;
constexpr auto kNarrow = dev::lora_fp8_kernel<1, 128, 72, 216, false>, kNarrowMerged = dev::lora_fp8_kernel<1, 128, 72, 216, true>;
inline auto kernel_of(int wide, int tile_n, int mixed) {
    if (wide) return mixed ? kWideApart : kWide;
    return tile_n == 256 ? (mixed ? kSingleMerged : kSingle) : mixed ? kNarrowMerged : kNarrow;
}
}  // namespace

size_t fp8_smem_bytes(int wide, int tile_n, int a_rows, int stages) {
    return 1024 + (size_t)stages * (a_rows + tile_n / (wide ? 2 : 1)) * kFp8StageRow + 8 * 64 * (wide ? 64 : 32) +
           2 * (512 / tile_n) * sizeof(dev::ScaleSlot) + 8 * (2 * (size_t)stages + 2 * 4 + 1) + 16;
}

static size_t shrink_smem_bytes(int n, int stages) {
    return 1024 + (size_t)stages * (kTileM + n) * kFp8StageRow + 8 * (2 * (size_t)stages + 2) + 16;
}
int shrink_stages(int n) {
    int s = 2;
    while (s < 8 && shrink_smem_bytes(n, s + 1) <= (size_t)kSmemLimit) ++s;
    return s;
}

cudaError_t launch_shrink(const ShrinkParams& p, int grid, cudaStream_t stream) {
    // the parts' sums take the rings' place: one unit a cluster
    const long long ctas = (long long)p.n_tiles * p.rank_tiles * p.parts;
    if (grid < 1 || grid > ctas || (p.parts > 1 && grid != ctas)) return cudaErrorInvalidValue;
    if (p.n < 16 || p.n > 256 || p.n % 16 || p.rank < 8 || p.rank % 8 || p.rank_tiles != (p.rank + p.n - 1) / p.n || p.parts < 1 || p.parts > kFp8MaxParts ||
        p.parts > p.k_steps || p.n_tiles < 1 || p.stages < 2 || shrink_smem_bytes(p.n, p.stages) > (size_t)kSmemLimit ||
        (p.parts > 1 && (size_t)p.stages * (kTileM + p.n) * kFp8StageRow < (size_t)p.n * kTileM * 4))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.dynamicSmemBytes = shrink_smem_bytes(p.n, p.stages);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)p.parts, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.chained ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, dev::lora_shrink_kernel, p);
}

cudaError_t fp8_prepare_device() {
    cudaError_t r = cudaFuncSetAttribute(dev::lora_shrink_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (r != cudaSuccess) return r;
    for (const auto k : {kWide, kWideApart, kSingle, kNarrow, kSingleMerged, kNarrowMerged}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

static void config(const Fp8Params& p, int grid, cudaStream_t stream, cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr /* [2] */) {
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = dim3(grid);
    cfg->blockDim = dim3(kFp8Threads);
    cfg->dynamicSmemBytes = fp8_smem_bytes(p.wide, p.tile_n, p.a_rows, p.stages);
    cfg->stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)(p.wide ? 2 : p.parts), 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = attr;
    cfg->numAttrs = p.chained ? 2 : 1;
}

// Clusters of `parts` CTAs of the single-CTA forms that the GPU holds at once.
int fp8_max_clusters(int tile_n, int parts) {
    Fp8Params p = {};
    p.tile_n = tile_n;
    p.parts = parts;
    p.a_rows = kTileM;
    p.stages = 3;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config(p, parts, nullptr, &cfg, attr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel_of(0, tile_n, 0), &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

int fp8_window(int bufs, int nk, int expands, int lora_stages) {
    int most = 0;
    for (int first = 0; first < nk + expands; ++first) {
        int sum = 0;
        for (int i = 0; i < bufs; ++i) sum += (first + i) % (nk + expands) < nk ? 1 : lora_stages;
        most = sum > most ? sum : most;
    }
    return most;
}

cudaError_t launch_fp8(const Fp8Params& p, int grid, cudaStream_t stream) {
    const int tile_rows = p.tile_n / (p.wide ? 2 : 1);
    if ((p.tile_n != 256 && (p.wide || p.tile_n != 128)) || p.parts < 1 || p.parts > kFp8MaxParts || p.parts > p.k_blocks ||
        (p.wide && (p.parts != 1 || p.a_rows != kTileM)) || p.a_rows < 16 || p.a_rows > kTileM || p.a_rows % 16)
        return cudaErrorInvalidValue;
    // stages: a lap is no shorter than the stages of the blocks between two uses of a TMEM buffer; an A stage's 128 rows lie
    // inside the rings; the parts' sums take the rings' place
    const size_t rings = (size_t)p.stages * (p.a_rows + tile_rows) * kFp8StageRow;
    if (p.lora_stages < 1 || p.k_lora % p.lora_stages || p.most_expands < 0 || p.expand_blocks != p.k_lora / p.lora_stages ||
        p.stages < fp8_window(512 / p.tile_n, p.k_blocks / p.parts, p.most_expands * p.expand_blocks, p.lora_stages) ||
        fp8_smem_bytes(p.wide, p.tile_n, p.a_rows, p.stages) > (size_t)kSmemLimit ||
        (size_t)p.stages * tile_rows < (size_t)(kTileM - p.a_rows) || (p.parts > 1 && rings < (size_t)p.tile_n * kTileM * 4))
        return cudaErrorInvalidValue;
    // units of K parts: one a cluster (the rings hold its sums at its end)
    const int span = p.wide ? 2 : p.parts;
    if (grid < 1 || grid % span || (p.parts > 1 && grid != p.n_groups * p.n_ntiles * p.parts)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config(p, grid, stream, &cfg, attr);
    return cudaLaunchKernelEx(&cfg, kernel_of(p.wide, p.tile_n, p.mixed), p);
}

}  // namespace lora
