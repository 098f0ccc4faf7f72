// Log probabilities of given tokens, with their ranks, the rows' entropies and the most likely tokens, in one pass over
// the logits:
//
//     z = x / temperature, m = max z, s = sum e^(z - m), lp_i = z_i - m - log s
//     entropy = log s - (1 / s) sum (z - m) e^(z - m)
//     rank of token t: the entries before it in the order of falling x, ties by rising index; the first `top` of that
//     order are the alternatives
//
// A row is a cluster of 1 to 8 CTAs' (one where there are rows enough), its parts joined through distributed shared
// memory: no workspace, no second launch, and the same order of sums in every run. Each thread keeps a running maximum
// and its two sums; a warp keeps the 32 largest entries that it has seen as 64-bit keys (value, then index), one a lane.
// Entries that may be among the first `top` are rare once the warp's own `top`-th and those of the block's other warps
// are known; they are collected in shared memory and merged 32 at a time.
//
// Bound by memory; 2-byte logits at the copy rate leave 11 lane instructions and 1.4 exponentials' time an entry.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dev_common.cuh"
#include "layer_internal.h"

namespace lora {
namespace {

constexpr int kWarps = 8, kThreadsScore = 32 * kWarps;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Order of entries as a 64-bit key: larger x first, then the smaller index; -0 is 0, a NaN is behind -inf. 0: none.
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
    if (k == 0) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(float x, int i) { return (uint64_t)ordered(x) << 32 | (uint32_t)~i; }
__device__ __forceinline__ float key_value(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) {
    return (uint64_t)__shfl_xor_sync(kAll, (uint32_t)(v >> 32), o) << 32 | __shfl_xor_sync(kAll, (uint32_t)v, o);
}
// Largest first over the lanes: a bitonic sort, and its last stage alone for a sequence that is bitonic already.
__device__ __forceinline__ uint64_t merge_step(uint64_t v, int o, bool up) {
    const uint64_t w = shfl_xor64(v, o);
    const bool low = ((threadIdx.x & o) == 0) == up;
    return low == (v > w) ? v : w;
}
__device__ __forceinline__ uint64_t sort32(uint64_t v) {
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
        for (int o = n >> 1; o; o >>= 1) v = merge_step(v, o, (threadIdx.x & n & 31) == 0);
    return v;
}
// The 32 largest of two sorted lists, sorted.
__device__ __forceinline__ uint64_t merge32(uint64_t a, uint64_t b) {
    const uint64_t r = shfl_xor64(b, 31);
    uint64_t v = a > r ? a : r;
#pragma unroll
    for (int o = 16; o; o >>= 1) v = merge_step(v, o, true);
    return v;
}

__device__ __forceinline__ float exp2_of(float t) {      // 2^-22 of the value; 0 below 2^-126
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}

// A part's sums: of 2^t and of t 2^t, t = (x - m) log2(e) / temperature; m = -inf: none yet.
struct Sums {
    float m, s, w;
};
__device__ __forceinline__ float from(float m) { return m == -INFINITY ? 0.f : m; }
// Both parts' sums under the larger maximum.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float c) {
    Sums r;
    r.m = fmaxf(a.m, b.m);
    const float base = from(r.m), ta = fmaxf((a.m - base) * c, -1000.f), tb = fmaxf((b.m - base) * c, -1000.f);
    const float ea = exp2_of(ta), eb = exp2_of(tb);
    r.s = a.s * ea + b.s * eb;
    r.w = (a.w + a.s * ta) * ea + (b.w + b.s * tb) * eb;
    return r;
}

struct Part {                          // of a CTA, or of a warp
    Sums sums;
    int ahead;                         // entries before the given token
};
struct Shared {
    uint64_t list[kWarps][32];
    uint64_t pending[kWarps][64];
    Part part[kWarps];
    uint64_t cta_list[32];
    Part cta_part;
    uint32_t bound;                    // the largest of the warps' `top`-th values, ordered
};

// A warp's 32 largest, and entries that wait to be merged into them.
struct Top {
    uint64_t mine;                     // this lane's of the list
    float own;                         // value of the list's `top`-th entry: a later entry has to be larger
    int count;                         // entries that wait
    bool full;                         // the list holds `top` entries
    __device__ __forceinline__ void merge(uint64_t* pending, int top, uint32_t* bound) {
        const int lane = threadIdx.x & 31;
        __syncwarp();
        uint64_t v = lane < count ? pending[lane] : 0;
        const uint64_t rest = lane + 32 < count ? pending[lane + 32] : 0;
        __syncwarp();
        pending[lane] = rest;
        count = max(0, count - 32);
        __syncwarp();
        mine = merge32(mine, sort32(v));
        const uint32_t hi = __shfl_sync(kAll, (uint32_t)(mine >> 32), top - 1);
        full = hi != 0;                // (a NaN's: any number is before it)
        own = unordered(hi);
        if (full && lane == 0) atomicMax(bound, hi);
    }
};

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Vec<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
};

template <typename T>
__global__ void __launch_bounds__(kThreadsScore) token_logprobs_kernel(const __grid_constant__ ScoreParams p) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int parts, part;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
    part = parts > 1 ? (int)dev::cluster_ctarank() : 0;
    const long long row = blockIdx.x / parts;
    if (tid == 0) sh.bound = 0;
    __syncthreads();
    dev::griddep_wait();
    dev::griddep_launch_dependents();

    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    const float c = p.inv_temperature * kLog2e;
    long long token = -1;
    if (p.tokens) token = p.tokens64 ? static_cast<const long long*>(p.tokens)[row] : static_cast<const int32_t*>(p.tokens)[row];
    const bool given = token >= 0 && token < p.vocab;
    const int tok = given ? (int)token : p.vocab;
    const float xt = given ? Vec<T>::one(x + tok) : INFINITY;
    const bool nan_token = xt != xt;

    // Entries [0, head) before the row's first 16-byte boundary (16 bytes: 8 or 4 entries), then vectors of 8, then the rest.
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T), p.vocab);
    const int n_vec = (p.vocab - head) >> 3, tail = head + 8 * n_vec;
    const int v0 = (int)((long long)n_vec * part / parts), v1 = (int)((long long)n_vec * (part + 1) / parts);

    Sums a = {-INFINITY, 0.f, 0.f};
    int ahead = 0;
    Top best = {0, 0.f, 0, false};
    float lane_bound = -INFINITY;          // no entry below it is among the warp's first `top`

    // Eight entries of this lane, the first at index i0; a missing one is -inf with no bit in `valid`. An entry equal to the
    // list's `top`-th is behind it, unless it was kept for the end (`late`).
    auto take = [&](const float* f, int i0, uint32_t valid, bool late) {
        float vm = fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
        if (vm > a.m) {
            const Sums none = {vm, 0.f, 0.f};
            a = join(a, none, c);
        }
        const float base = from(a.m);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float t = (f[k] - base) * c, e = exp2_of(t);
            a.s += e;
            a.w = fmaf(e, fmaxf(t, -1000.f), a.w);             // (0 for -inf; a NaN is in e)
        }
        if (nan_token) {
#pragma unroll
            for (int k = 0; k < 8; ++k) ahead += (valid >> k & 1) && (f[k] == f[k] || i0 + k < tok);
        } else if (vm >= xt) {
            if (i0 + 8 <= tok) {
#pragma unroll
                for (int k = 0; k < 8; ++k) ahead += f[k] >= xt && (valid >> k & 1);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) ahead += f[k] > xt || (f[k] == xt && i0 + k < tok && (valid >> k & 1));
            }
        }
        if (p.top == 0) return;                                // (the whole warp)
        const float least = fmaxf(lane_bound, unordered(max(*const_cast<volatile uint32_t*>(&sh.bound), 0x007fffffu)));
        uint32_t pass = 0;
        if (!best.full || late || (vm > best.own && vm >= least)) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                pass |= (uint32_t)(!best.full || late ? !(f[k] < least) : f[k] > best.own && f[k] >= least) << k;
            pass &= valid;
        }
        if (!__any_sync(kAll, pass)) return;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            const uint32_t who = __ballot_sync(kAll, pass >> k & 1);
            if (!who) continue;
            float v = f[0];                                    // (f[k] without an array in memory)
#pragma unroll
            for (int j = 1; j < 8; ++j) v = j == k ? f[j] : v;
            if (pass >> k & 1) sh.pending[warp][best.count + __popc(who & ((1u << lane) - 1))] = key_of(v, i0 + k);
            best.count += __popc(who);
            if (best.count >= 32) best.merge(sh.pending[warp], p.top, &sh.bound);
        }
    };

    constexpr int N = 4;                                       // vectors in flight
    const T* xv = x + head;
    for (int v = v0 + warp * 32; v < v1; v += N * kThreadsScore) {
        Vec<T> u[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = v + i * kThreadsScore + lane;
            if (at < v1) u[i].load(xv + 8ll * at);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = v + i * kThreadsScore + lane;
            if (v + i * kThreadsScore >= v1) break;
            float f[8];
            if (at < v1) {
                u[i].get(f);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = -INFINITY;
            }
            if (p.top && lane_bound == -INFINITY && !best.full && at - lane + 32 <= v1) {
                // the warp's first vectors: `top` lanes have a largest entry of at least the `top`-th of those
                const float vm = fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
                const uint32_t hi = (uint32_t)(sort32((uint64_t)ordered(vm) << 32 | lane) >> 32);
                lane_bound = fmaxf(unordered(__shfl_sync(kAll, hi, p.top - 1)), -INFINITY);
            }
            take(f, head + 8 * at, at < v1 ? 0xffu : 0u, false);
        }
    }
    // The head and the tail: one entry a lane, of the first part's first warp.
    if (part == 0 && warp == 0) {
        const int n = p.vocab - tail, i = lane < head ? lane : lane - 16 >= 0 && lane - 16 < n ? tail + lane - 16 : -1;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = -INFINITY;
        if (i >= 0) f[0] = Vec<T>::one(x + i);
        take(f, i >= 0 ? i : 0, i >= 0 ? 1u : 0u, true);
    }
    if (p.top)
        while (best.count) best.merge(sh.pending[warp], p.top, &sh.bound);

    // the warp's sums, then the block's, then the cluster's
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Sums b = {__shfl_xor_sync(kAll, a.m, o), __shfl_xor_sync(kAll, a.s, o), __shfl_xor_sync(kAll, a.w, o)};
        // (the lower lane's first in both, so that both have the same bits)
        a = lane & o ? join(b, a, c) : join(a, b, c);
        ahead += __shfl_xor_sync(kAll, ahead, o);
    }
    sh.list[warp][lane] = best.mine;
    if (lane == 0) sh.part[warp] = Part{a, ahead};
    __syncthreads();
    if (warp == 0) {
        uint64_t v = best.mine;
        for (int i = 1; i < kWarps; ++i) {
            a = join(a, sh.part[i].sums, c);
            ahead += sh.part[i].ahead;
            if (p.top) v = merge32(v, sh.list[i][lane]);
        }
        best.mine = v;
        sh.cta_list[lane] = v;
        if (lane == 0) sh.cta_part = Part{a, ahead};
    }
    if (parts > 1) {
        dev::cluster_sync();
        if (part == 0 && warp == 0) {
            const uint32_t list = dev::smem_addr(&sh.cta_list[lane]), from_part = dev::smem_addr(&sh.cta_part);
            for (int i = 1; i < parts; ++i) {
                Part b;
                uint64_t v;
                const uint32_t pa = dev::map_to_rank(from_part, (uint32_t)i);
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(dev::map_to_rank(list, (uint32_t)i)) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.sums.m) : "r"(pa) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1+4];" : "=f"(b.sums.s) : "r"(pa) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1+8];" : "=f"(b.sums.w) : "r"(pa) : "memory");
                asm volatile("ld.shared::cluster.u32 %0, [%1+12];" : "=r"(b.ahead) : "r"(pa) : "memory");
                a = join(a, b.sums, c);
                ahead += b.ahead;
                if (p.top) best.mine = merge32(best.mine, v);
            }
        }
        dev::cluster_sync();                                   // the parts have been read
    }
    if (part != 0 || warp != 0) return;
    const float log_s = logf(a.s);                             // (a row of -inf alone: log 0)
    auto lp = [&](float v) { return v == -INFINITY && a.s == a.s ? v : (v - from(a.m)) * p.inv_temperature - log_s; };
    if (lane == 0) {
        if (p.entropy) p.entropy[row] = a.s == 0.f ? 0.f : log_s - kLn2 * a.w / a.s;
        if (p.logprobs) p.logprobs[row] = given ? lp(xt) : __uint_as_float(0x7fc00000u);
        if (p.ranks) p.ranks[row] = given ? ahead : -1;
    }
    if (lane < p.top) {
        p.top_logprobs[row * p.top + lane] = lp(key_value(best.mine));
        p.top_tokens[row * p.top + lane] = key_index(best.mine);
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const ScoreParams& p, cudaStream_t stream) {
    // A cluster a row while rows are few: half of the GPU's room for blocks (four an SM) filled, and parts of at least
    // 2,048 entries.
    int parts = 1;
    while (parts < 8 && (long long)p.rows * parts * 2 <= 608 && p.vocab / (parts * 2) >= 2048) parts *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)parts, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows * parts);
    cfg.blockDim = dim3(kThreadsScore);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return p.is_fp32 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<float>, p)
                     : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<__nv_bfloat16>, p);
}

}  // namespace lora
