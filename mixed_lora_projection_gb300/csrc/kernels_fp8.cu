// sm_103a kernel of the projection with 8-bit activations and an 8-bit base weight:
//
//     acc[t, n]  = sum_g xs[t, g] ws[n / 128, g] sum_{k in group g} X[t, k] W[n, k]
//     acc[t, n] += U[t, :] B_a[n, :]^T        (adapter tiles; U from the bf16 shrink before this launch)
//     Y[t, n]    = bf16(acc[t, n])
//
// A group's 128 products are summed by tcgen05.mma kind::f8f6f4 in tensor memory; each group has a scale of
// its own per row and block of columns, so its sums leave tensor memory and are added, times that scale, to
// fp32 accumulators in the epilogue warps' registers. The expand is one more such block (kind::f16, bf16
// operands, all of the rank) with scale 1.
//
// Per CTA: warp 0 loads the stages (TMA, rows of 128 bytes, 128-byte swizzle: 128 e4m3 or 64 bf16); warps 1 and
// 2 issue the even and the odd blocks' MMAs into the two TMEM buffers (a warp's barrier wait completes after the
// MMAs that it issued, so one warp's waits run under the other's MMAs); warp 3 owns TMEM; warps 4..11 are the
// epilogue, two per TMEM lane quadrant, half of the columns each.
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

// The blocks of one unit as every role walks them: base groups [kb0, kb0 + nk), then the expand's block.
struct Work {
    Tile tile;
    int n0, kb0, nk, expand;
};
template <int CG>
__device__ __forceinline__ Work decode(const Fp8Params& p, const Tile* tiles, int u, int rank, int part) {
    Work w;
    const int per = p.n_groups * p.raster_group;
    const int g = u / per, r = u - g * per;
    const int gw = min(p.raster_group, p.n_ntiles - g * p.raster_group);
    w.tile = tiles[(r / gw) * CG + rank];
    w.n0 = (g * p.raster_group + r % gw) * p.tile_n;
    w.kb0 = part * p.k_blocks / p.parts;
    w.nk = (part + 1) * p.k_blocks / p.parts - w.kb0;
    w.expand = w.tile.adapter && part == p.parts - 1;
    return w;
}

// NT: columns of a TMEM buffer, NT / 2 of them in each epilogue thread's registers. Registers of the launch are
// dealt out anew: the loading warps' to the epilogue's accumulators (LOW x 128 + HIGH x 256 <= 384 x the launch's).
template <int CG, int NT, int BLOCKS, int LOW, int HIGH>
__global__ void __launch_bounds__(kFp8Threads, BLOCKS) lora_fp8_kernel(const __grid_constant__ Fp8Params p) {
    static_assert(CG == 1 || NT == 256, "SM pairs run 256-column blocks");
    constexpr int kHalf = NT / 2, kChunks = kHalf / 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int stages = p.stages;
    const uint32_t a_bytes = (uint32_t)p.a_rows * kFp8StageRow;
    const uint32_t b_bytes = (uint32_t)(p.tile_n / CG) * kFp8StageRow;
    // an A stage of fewer than 128 rows: the MMA's other rows read what follows in the rings, and are never stored
    uint8_t* a_ring = base;
    uint8_t* b_ring = a_ring + (size_t)stages * a_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(b_ring + (size_t)stages * b_bytes);
    uint64_t* empty = full + stages;
    uint64_t* tfull = empty + stages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&tfull[b]), 1);
            mbar_init(smem_addr(&tempty[b]), CG * 8);
        }
        mbar_init(smem_addr(drain), 2);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3) tmem_alloc<CG>(smem_addr(tmem_slot), 2 * NT);
    tc_fence_before();
    if (CG > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t limit = p.wait_limit_ns;
    const Tile* tiles = p.inline_wl ? p.inline_tiles : p.tiles;
    const CUtensorMap* bmaps = p.inline_wl ? p.inline_bmaps : p.tm_b;
    griddep_wait();
    griddep_launch_dependents();

    if (warp < 4) {
        regs_dec<LOW>();
        const uint32_t issuer = lane == 0 ? 1u : 0u;
        if (warp == 0 && !p.debug_stall) {
            // ------------------------------------------------------------ TMA producer (lane 0 issues)
            int stage = 0, issued = 0, acquired = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t tx = CG * (a_bytes + b_bytes);
            for (int u = first; u < n_units && ok; u += step) {
                const Work w = decode<CG>(p, tiles, u, rank, part);
                const int nb = w.nk + (w.expand ? p.k_lora : 0);
                const CUtensorMap* bm = &bmaps[w.expand ? w.tile.adapter - 1 : 0];
                if (w.expand && !p.inline_wl && acquired != w.tile.adapter) {
                    tensormap_acquire(bm);
                    acquired = w.tile.adapter;
                }
                for (int b = 0; b < nb; ++b) {
                    if (!wait_all(smem_addr(&empty[stage]), phase ^ 1, abort_flag, p.status, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_addr(&full[stage]);
                    mbar_arrive_expect_tx(bar, tx, leader ? issuer : 0u);
                    const uint32_t fb = CG > 1 ? map_to_rank(bar, 0) : bar;
                    const uint32_t sa = smem_addr(a_ring + (size_t)stage * a_bytes), sb = smem_addr(b_ring + (size_t)stage * b_bytes);
                    const bool main = b < w.nk;
                    const int k = main ? (w.kb0 + b) * kFp8Group : (b - w.nk) * 64;
                    tma_load_2d<CG>(sa, main ? &p.tm_x : &p.tm_u, fb, k, main ? w.tile.row0 : w.tile.u_row, issuer);
                    tma_load_2d<CG>(sb, main ? &p.tm_w : bm, fb, k, w.n0 + rank * (p.tile_n / CG), issuer);
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
            const uint32_t idesc8 = instr_desc_e4m3(kTileM * CG, p.tile_n), idesc16 = instr_desc_bf16(kTileM * CG, p.tile_n);
            const int mine = warp - 1;                       // parity of the blocks this warp issues, and their buffer
            const uint32_t d = tmem_base + (uint32_t)(mine * NT);
            int stage = 0, blk = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = first; u < n_units && ok; u += step) {
                const Work w = decode<CG>(p, tiles, u, rank, part);
                const int nb = w.nk + w.expand;
                for (int b = 0; b < nb; ++b, ++blk) {
                    const bool main = b < w.nk;
                    const int ns = main ? 1 : p.k_lora;
                    const bool act = (blk & 1) == mine;
                    if (act && !wait_all(smem_addr(&tempty[mine]), ((blk >> 1) & 1) ^ 1, abort_flag, p.status, limit)) {
                        ok = false;
                        break;
                    }
                    for (int s = 0; s < ns; ++s) {
                        if (act) {
                            if (!wait_all(smem_addr(&full[stage]), phase, abort_flag, p.status, limit)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t ad = smem_desc<64>(smem_addr(a_ring + (size_t)stage * a_bytes));
                            const uint64_t bd = smem_desc<64>(smem_addr(b_ring + (size_t)stage * b_bytes));
                            // 32 bytes along K inside the swizzled rows a step
                            if (main) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_e4m3<CG>(d, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), idesc8, k > 0 ? 1u : 0u, issuer);
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_bf16<CG>(d, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), idesc16, (s > 0 || k > 0) ? 1u : 0u,
                                                 issuer);
                            }
                            mma_commit<CG>(smem_addr(&empty[stage]), issuer);
                        }
                        if (++stage == stages) { stage = 0; phase ^= 1; }
                    }
                    if (!ok) break;
                    if (act) mma_commit<CG>(smem_addr(&tfull[mine]), issuer);
                }
            }
            // every MMA this warp issued has completed before TMEM is released
            mma_commit_local<CG>(smem_addr(drain), issuer);
            if (lane == 0) wait_lane(smem_addr(drain), 0, abort_flag, p.status, limit, false);
        }
        __syncwarp();
        if (CG == 1 && p.parts > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        // ------------------------------------------------------------ epilogue
        regs_inc<HIGH>();
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int r_local = q * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        const int cols = CG > 1 ? kHalf : p.tile_n >> 1;     // of this thread: a multiple of 16
        const int nblk = (p.d_out + kFp8Group - 1) / kFp8Group;
        int blk = 0;
        bool ok = true;
        for (int u = first; u < n_units && ok; u += step) {
            const Work w = decode<CG>(p, tiles, u, rank, part);
            const int row = w.tile.row0 + r_local;
            const bool row_ok = r_local < w.tile.nrows;
            const int c0 = w.n0 + half * cols;
            // the thread's columns lie in at most two blocks of 128 output features
            const int b0 = min(c0 >> 7, nblk - 1), b1 = min((c0 + cols - 1) >> 7, nblk - 1);
            const float* xs = p.xs + (long long)(row_ok ? row : w.tile.row0) * p.k_blocks + w.kb0;
            const float* ws0 = p.ws + (long long)b0 * p.k_blocks + w.kb0;
            const float* ws1 = p.ws + (long long)b1 * p.k_blocks + w.kb0;
            const int cut = (((c0 >> 7) + 1) << 7) - c0;     // columns before the second block's
            const bool any = w.tile.nrows > 0;
            uint64_t acc[kHalf / 2];
#pragma unroll
            for (int i = 0; i < kHalf / 2; ++i) acc[i] = 0;
            const int nb = w.nk + w.expand;
            float sx = 0.f, s0 = 0.f, s1 = 0.f;
            if (any && w.nk > 0) { sx = __ldg(xs); s0 = __ldg(ws0); s1 = __ldg(ws1); }
            for (int b = 0; b < nb; ++b, ++blk) {
                float f0 = sx * s0, f1 = sx * s1;
                if (b >= w.nk) f0 = f1 = 1.f;
                if (any && b + 1 < w.nk) {                   // the next block's scales, under this one's wait
                    sx = __ldg(xs + b + 1);
                    s0 = __ldg(ws0 + b + 1);
                    s1 = __ldg(ws1 + b + 1);
                }
                const int buf = blk & 1;
                if (!wait_all(smem_addr(&tfull[buf]), (blk >> 1) & 1, abort_flag, p.status, limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t = tmem_base + (uint32_t)(buf * NT + half * cols) + lane_off;
                const uint64_t g0 = pair(__float_as_uint(f0), __float_as_uint(f0)), g1 = pair(__float_as_uint(f1), __float_as_uint(f1));
                if (CG > 1) {                                // the next columns' load runs under this one's sums
                    uint32_t v[2][16];
                    tmem_ld16(t, v[0]);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        tmem_wait16(v[c & 1]);
                        if (c + 1 < kChunks) tmem_ld16(t + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[8 * c + i] = fma2(pair(v[c & 1][2 * i], v[c & 1][2 * i + 1]), g0, acc[8 * c + i]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        if (16 * c < cols) {
                            uint32_t v[16];
                            tmem_ld16(t + 16 * c, v);
                            tmem_wait16(v);
                            const uint64_t g = 16 * c < cut ? g0 : g1;
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[8 * c + i] = fma2(pair(v[2 * i], v[2 * i + 1]), g, acc[8 * c + i]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG > 1) mbar_arrive_cluster(map_to_rank(smem_addr(&tempty[buf]), 0));
                    else mbar_arrive(smem_addr(&tempty[buf]));
                }
            }
            if (!ok) break;
            if (CG > 1 || p.parts == 1) {
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.y) + (long long)row * p.d_out + c0;
                if (row_ok) {
#pragma unroll
                    for (int c = 0; c < kHalf / 8; ++c) {
                        if (8 * c < cols && c0 + 8 * c < p.d_out) {
                            uint4 o;
                            o.x = pack_bf16x2(lo2(acc[4 * c]), hi2(acc[4 * c]));
                            o.y = pack_bf16x2(lo2(acc[4 * c + 1]), hi2(acc[4 * c + 1]));
                            o.z = pack_bf16x2(lo2(acc[4 * c + 2]), hi2(acc[4 * c + 2]));
                            o.w = pack_bf16x2(lo2(acc[4 * c + 3]), hi2(acc[4 * c + 3]));
                            *reinterpret_cast<uint4*>(out + 8 * c) = o;
                        }
                    }
                }
            } else {
                // every stage has been read (the MMAs' commits): this part's sums take the rings' place, four
                // columns of the 128 rows side by side
                float4* sums = reinterpret_cast<float4*>(base);
#pragma unroll
                for (int c = 0; c < kHalf / 4; ++c)
                    if (4 * c < cols)
                        sums[(half * (cols >> 2) + c) * 128 + r_local] =
                            make_float4(lo2(acc[2 * c]), hi2(acc[2 * c]), lo2(acc[2 * c + 1]), hi2(acc[2 * c + 1]));
            }
        }
        if (CG == 1 && p.parts > 1) {
            cluster_sync();
            if (ok) {
                // each CTA adds its share of the columns over the parts, in their order
                const Work w = decode<CG>(p, tiles, first, rank, part);
                const int per = p.tile_n / p.parts, vecs = per >> 3, t = (int)threadIdx.x - 128;
                for (int i = t; i < w.tile.nrows * vecs; i += 256) {
                    const int r = i / vecs, c = part * per + 8 * (i - r * vecs);
                    if (w.n0 + c >= p.d_out) continue;
                    float s[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[k] = 0.f;
                    const uint32_t at = smem_addr(base) + (uint32_t)(((c >> 2) * 128 + r) * 16);
                    for (int j = 0; j < p.parts; ++j) {
                        const uint32_t a = map_to_rank(at, (uint32_t)j);
                        const float4 x = ld_cluster(a), y = ld_cluster(a + 128 * 16);
                        s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
                        s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
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
        tmem_dealloc<CG>(tmem_base, 2 * NT);
    }
}

}  // namespace
}  // namespace dev

namespace {
constexpr auto kNarrow = dev::lora_fp8_kernel<1, 128, 2, 32, 104>;
constexpr auto kWide = dev::lora_fp8_kernel<2, 256, 1, 40, 232>;
}  // namespace

size_t fp8_smem_bytes(int tile_rows, int a_rows, int stages) {
    return 1024 + (size_t)stages * (a_rows + tile_rows) * kFp8StageRow + 8 * (2 * (size_t)stages + 5) + 16;
}

cudaError_t fp8_prepare_device() {
    const cudaError_t e = cudaFuncSetAttribute(kNarrow, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(kWide, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
}

cudaError_t launch_fp8(const Fp8Params& p, int grid, cudaStream_t stream) {
    const int cg = p.wide ? 2 : 1, tile_rows = p.tile_n / cg;
    const size_t smem = fp8_smem_bytes(tile_rows, p.a_rows, p.stages);
    if (p.wide ? (p.tile_n != 256 || p.parts != 1 || p.a_rows != kTileM)
               : (p.tile_n < 32 || p.tile_n > 128 || p.tile_n % 32 || p.parts < 1 || p.parts > kFp8MaxParts || p.tile_n % (8 * p.parts)))
        return cudaErrorInvalidValue;
    // an A stage's 128 rows lie inside the rings; the parts' sums (parts > 1) take the rings' place
    const size_t rings = (size_t)p.stages * (p.a_rows + tile_rows) * kFp8StageRow;
    if (p.stages < 2 || smem > (size_t)kSmemLimit || p.a_rows < 16 || p.a_rows > kTileM || p.a_rows % 16 ||
        (size_t)p.stages * tile_rows * kFp8StageRow < (size_t)(kTileM - p.a_rows) * kFp8StageRow ||
        (p.parts > 1 && rings < (size_t)p.tile_n * kTileM * 4) || grid < 1 || grid % (cg * p.parts) ||
        (!p.wide && grid != p.n_groups * p.n_ntiles * p.parts))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFp8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)(cg * p.parts), 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, p.wide ? kWide : kNarrow, p);
}

}  // namespace lora
