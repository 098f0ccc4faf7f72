// Log probabilities of given tokens, with their ranks, the rows' entropies and the most likely tokens, in one pass over
// the logits:
//
//     z = x / temperature, m = max z, s = sum e^(z - m), lp_i = z_i - m - log s
//     entropy = log s - (1 / s) sum (z - m) e^(z - m)        (any reference m gives the same; in base 2 below)
//     rank of token t: the entries before it in the order of falling x, ties by rising index; the first `top` of that
//     order are the alternatives
//
// A row is a cluster's of 1 to 8 CTAs (one where there are rows enough), its parts joined through distributed shared
// memory: no workspace, no second launch, and the same order of sums in every run. Each thread keeps a reference and its
// two sums. Vectors of eight entries that may hold some of the first `top` wait as 64-bit keys (their largest entry, their
// index) in columns of the lanes' own: every lane knows its largest entry, a warp the share-th largest of its lanes'
// (share = top over the warps, rounded up; a few warp reductions), and no entry below the smallest of the warps' is among
// the CTA's first `top`. That leaves some 150 vectors of 100,000 entries for `top` 20. The first `top` of them hold the
// first `top` entries; they are read once more, and a key's place is the number of larger ones.
//
// 2-byte logits at the copy rate leave 11 lane instructions and 1.4 exponentials' time an entry; bound by the
// instructions (nine an entry, thirteen with alternatives; 68 and 72 % of the issue slots used). 4,096 rows of 100,003 in
// bf16: 156 us (5.3 TB/s), with 20 alternatives 209; 2,048 rows of 131,072 in fp32 168 (6.4 TB/s) and 208. Collecting by
// a ballot and a shared count took 238 of those 209 us. Loads through shared memory (cp.async, four deep, in place of the
// next iteration's in registers) took 248 and, in fp32, 264 for 168.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dev_common.cuh"
#include "layer_internal.h"

namespace lora {
namespace {

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

// A part's sums: of 2^t and of t 2^t, t = (x - m) log2(e) / temperature; the reference m is an entry; -inf: none yet.
struct Sums {
    float m, s, w;
};
__device__ __forceinline__ float from(float m) { return m == -INFINITY ? 0.f : m; }
// Both parts' sums from the larger reference.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float c) {
    Sums j;
    j.m = fmaxf(a.m, b.m);
    const float base = from(j.m), ta = fmaxf((a.m - base) * c, -1000.f), tb = fmaxf((b.m - base) * c, -1000.f);
    const float ea = exp2_of(ta), eb = exp2_of(tb);
    j.s = a.s * ea + b.s * eb;
    j.w = (a.w + a.s * ta) * ea + (b.w + b.s * tb) * eb;
    return j;
}

struct Part {                          // of a CTA, or of a warp
    Sums sums;
    int ahead;                         // entries before the given token
};
// Vectors that a lane may have waiting: 8, what four iterations add, and the head or the tail.
constexpr int kSettle = 8, kPending = kSettle + 2 * 4 + 1;
template <int WARPS>
struct Shared {
    alignas(16) uint64_t pending[WARPS][kPending * 32];   // a warp's: its lanes' first, then their second, ...
    alignas(16) uint64_t pool[256];    // what the warps, or the cluster's CTAs, bring to the last choice
    uint64_t list[32];                 // its outcome
    Part part[WARPS];
    float bound[WARPS];                // at least `share` entries of the warp are as large
    int pooled;
    Part cta_part;
};

// A vector as it waits: its largest entry's bits, then its index.
__device__ __forceinline__ uint64_t ordered_key(uint64_t k) { return key_of(__uint_as_float((uint32_t)(k >> 32)), (int)(uint32_t)k); }

// A warp's waiting vectors, n of this lane's, without those below `floor`, at most its 32 first: to the front of
// `pending`. Returns how many are left; plus 64 where there were more, then they are sorted.
__device__ __noinline__ int settle(uint64_t* pending, int n, uint64_t floor) {
    const int lane = threadIdx.x & 31, most = __reduce_max_sync(kAll, n);
    int left = 0;
    __syncwarp();
    for (int i = 0; i < most; ++i) {                           // (in place: what moves goes down)
        const uint64_t w = i < n ? pending[32 * i + lane] : 0;
        const uint32_t keep = __ballot_sync(kAll, i < n && ordered_key(w) >= floor);
        __syncwarp();
        if (keep >> lane & 1) pending[left + __popc(keep & ((1u << lane) - 1))] = w;
        __syncwarp();
        left += __popc(keep);
    }
    if (left <= 32) return left;
    uint64_t best = 0;
    for (int i = 0; i < left; i += 32) best = merge32(best, sort32(i + lane < left ? ordered_key(pending[i + lane]) : 0));
    __syncwarp();
    pending[lane] = (uint64_t)__float_as_uint(key_value(best)) << 32 | (uint32_t)key_index(best);
    __syncwarp();
    return 32 + 64;
}

// The pool, its count and the last list, before keys are brought to it. All threads.
template <int WARPS>
__device__ __forceinline__ void clear(Shared<WARPS>& sh) {
    __syncthreads();                                           // they have been read
    if (threadIdx.x == 0) sh.pooled = 0;
    if (threadIdx.x < 32) sh.list[threadIdx.x] = 0;
    __syncthreads();
}
// Every lane's key, where it has one (not 0), to the pool, side by side.
template <int WARPS>
__device__ __forceinline__ void bring(Shared<WARPS>& sh, uint64_t key) {
    const int lane = threadIdx.x & 31;
    const uint32_t have = __ballot_sync(kAll, key != 0);
    int at = 0;
    if (lane == 0 && have) at = atomicAdd(&sh.pooled, __popc(have));
    at = __shfl_sync(kAll, at, 0);
    if (key) sh.pool[at + __popc(have & ((1u << lane) - 1))] = key;
}

// The first `top` of the keys in the pool, in their order, to sh.list: a key's place is the number of larger ones. All
// threads; sh.list is theirs to read after a barrier.
template <int WARPS>
__device__ __forceinline__ void choose(Shared<WARPS>& sh, int top) {
    __syncthreads();
    const int n = sh.pooled;
    for (int i = threadIdx.x; i < n; i += 32 * WARPS) {
        const uint64_t mine = sh.pool[i];
        int place = 0;
        const ulonglong2* all = reinterpret_cast<const ulonglong2*>(sh.pool);
#pragma unroll 4
        for (int j = 0; j < n / 2; ++j) {
            const ulonglong2 k = all[j];
            place += (k.x > mine) + (k.y > mine);
        }
        if (n & 1) place += sh.pool[n - 1] > mine;
        if (place < top && mine) sh.list[place] = mine;        // (0: none; keys differ by their index)
    }
}

// Two fp32 values in one instruction.
__device__ __forceinline__ uint64_t two(float x, float y) { return (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x); }
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void none() { u = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }   // -inf
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
    __device__ __forceinline__ void none() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
};
__device__ __forceinline__ float max3(float a, float b, float c) {      // (a NaN counts as none)
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ float max8(const float* f) { return max3(max3(f[0], f[1], f[2]), max3(f[3], f[4], f[5]), fmaxf(f[6], f[7])); }

// A thread's pass over its vectors of 8 entries.
template <typename T, int WARPS>
struct Pass {
    const ScoreParams& p;
    Shared<WARPS>& sh;
    float c, xt;                       // log2(e) / temperature; the given token's logit
    int tok;
    bool nan_token;
    uint64_t c2, base2;                // c, and minus the reference, twice each
    float limit;                       // an entry over it moves the reference; -inf: no reference yet
    uint64_t s2, w2;                   // both sums, of even and of odd entries
    int ahead;
    float largest;                     // of this lane's entries
    float bound;                       // at least `top` entries of the CTA are as large: no smaller one is among its first
    uint64_t own;                      // the warp's top-th largest key, once it has sorted its keys: no vector behind it
                                       // is wanted either (0: not sorted yet)
    float least;                       // by both: a vector without an entry as large is not wanted
    int waiting;                       // this lane's vectors in sh.pending

    __device__ __forceinline__ Pass(const ScoreParams& p, Shared<WARPS>& sh) : p(p), sh(sh) {}

    // Sums of eight entries. The reference stays while no entry is more than 2^8 times its weight (an exponent's rounding
    // then stays below 2^-21), so that it moves a few times a row and not with every new maximum.
    __device__ __forceinline__ void sum(const float* f, float vm) {
        if (vm > limit) {
            const float m = limit == -INFINITY ? -INFINITY : -lo2(base2), ta = fmaxf((m - vm) * c, -1000.f), ea = exp2_of(ta);
            w2 = mul2(fma2(s2, two(ta, ta), w2), two(ea, ea));
            s2 = mul2(s2, two(ea, ea));
            base2 = two(-vm, -vm);
            limit = vm + 8.f / c;
        }
        uint64_t t[4], e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            t[k] = mul2(add2(two(f[2 * k], f[2 * k + 1]), base2), c2);
            e[k] = two(exp2_of(lo2(t[k])), exp2_of(hi2(t[k])));
            s2 = add2(s2, e[k]);
        }
        uint64_t w = w2;
#pragma unroll
        for (int k = 0; k < 4; ++k) w = fma2(e[k], t[k], w);
        const float both = lo2(w) + hi2(w);
        if (both != both) {                                    // an entry of -inf, of weight 0 (a NaN is in its exponential too)
            w = w2;
#pragma unroll
            for (int k = 0; k < 4; ++k) w = fma2(e[k], two(fmaxf(lo2(t[k]), -1000.f), fmaxf(hi2(t[k]), -1000.f)), w);
        }
        w2 = w;
    }
    __device__ __forceinline__ float weights() const { return lo2(s2) + hi2(s2); }
    __device__ __forceinline__ Sums sums() const { return Sums{limit == -INFINITY ? -INFINITY : -lo2(base2), weights(), lo2(w2) + hi2(w2)}; }

    // Entries before the given token among eight, the first at index i0.
    __device__ __forceinline__ void count(const float* f, float vm, int i0, uint32_t valid) {
        if (nan_token) {
#pragma unroll
            for (int k = 0; k < 8; ++k) ahead += (valid >> k & 1) && (f[k] == f[k] || i0 + k < tok);
        } else if (vm >= xt) {
            if (i0 + 8 <= tok && valid == 0xff) {
#pragma unroll
                for (int k = 0; k < 8; ++k) ahead += f[k] >= xt;
            } else if (i0 > tok) {
#pragma unroll
                for (int k = 0; k < 8; ++k) ahead += f[k] > xt;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) ahead += f[k] > xt || (f[k] == xt && i0 + k < tok && (valid >> k & 1));
            }
        }
    }

    // Whether a vector, its largest entry vm, may hold some of the first `top`; NaNs, in vectors that hold nothing else, as
    // well: they are among them where there are fewer numbers.
    __device__ __forceinline__ bool wanted(float vm) const { return !(vm < least); }
    __device__ __forceinline__ void push(float vm, int vector) {
        sh.pending[threadIdx.x >> 5][32 * waiting + (threadIdx.x & 31)] = (uint64_t)__float_as_uint(vm) << 32 | (uint32_t)vector;
        ++waiting;
    }
    __device__ __forceinline__ int settled() {
        return settle(sh.pending[threadIdx.x >> 5], waiting, (uint64_t)(bound == -INFINITY ? 0 : ordered(bound)) << 32);
    }
    // Where a lane has much waiting, the warp keeps its 32 first: the first `top` entries are in the `top` first vectors.
    __device__ __forceinline__ void thin() {
        const int left = settled();
        if (left >= 64) {
            own = ordered_key(sh.pending[threadIdx.x >> 5][p.top - 1]);
            raise();
        }
        __syncwarp();
        waiting = (threadIdx.x & 31) < (left & 63);
    }
    // (a vector equal to the warp's top-th comes behind it: a warp's vectors come in rising order)
    __device__ __forceinline__ void raise() {
        const uint32_t hi = (uint32_t)(own >> 32);
        least = fmaxf(bound, hi ? unordered(hi + 1) : -INFINITY);
    }
    // The warp's share-th largest of its lanes' largest entries.
    __device__ __forceinline__ void mark(int share) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        uint32_t v = ordered(largest), m = 0;
        for (int i = 0; i < share; ++i) {
            m = __reduce_max_sync(kAll, v);
            if (lane == __ffs(__ballot_sync(kAll, v == m)) - 1) v = 0;
        }
        if (lane == 0 && m) sh.bound[warp] = unordered(m);
    }
    __device__ __forceinline__ void renew() {
        float b = *const_cast<volatile float*>(&sh.bound[0]);
#pragma unroll
        for (int i = 1; i < WARPS; ++i) b = fminf(b, *const_cast<volatile float*>(&sh.bound[i]));
        bound = b;
        raise();
    }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename T, bool TOP, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS) token_logprobs_kernel(const __grid_constant__ ScoreParams p) {
    constexpr int kThreads = 32 * WARPS;
    __shared__ Shared<WARPS> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int parts, part;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
    part = parts > 1 ? (int)dev::cluster_ctarank() : 0;
    const long long row = blockIdx.x / parts;
    if (tid < 32) sh.list[tid] = 0;
    if (tid == 0) sh.pooled = 0;
    if (tid < WARPS) sh.bound[tid] = -INFINITY;
    dev::griddep_wait();
    dev::griddep_launch_dependents();

    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    // Entries [0, head) before the row's first 16-byte boundary, then vectors of 8, then the rest.
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T), p.vocab);
    const int n_vec = (p.vocab - head) >> 3, tail = head + 8 * n_vec;
    const int v0 = (int)((long long)n_vec * part / parts), v1 = (int)((long long)n_vec * (part + 1) / parts);
    const T* xv = x + head;
    // (few rows: a thread's loads of one iteration would wait for the last one's, a memory's latency each)
    if (WARPS == 8 && parts > 1 && tid == 0 && v1 > v0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(xv + 8ll * v0), "r"((uint32_t)min((long long)(v1 - v0) * 8 * (int)sizeof(T), 1ll << 18)) : "memory");

    // Two vectors an iteration, the next two in flight; a vector that is not there is one of -inf.
    Vec<T> u0, u1;
    auto load = [&](int at) {
        if (at - tid + 2 * kThreads <= v1) {                   // (all of the CTA's)
            u0.load(xv + 8ll * at);
            u1.load(xv + 8ll * (at + kThreads));
            return;
        }
        u0.none();
        u1.none();
        if (at < v1) u0.load(xv + 8ll * at);
        if (at + kThreads < v1) u1.load(xv + 8ll * (at + kThreads));
    };
    int at = v0 + tid;
    load(at);
    long long token = -1;
    if (p.tokens) token = p.tokens64 ? static_cast<const long long*>(p.tokens)[row] : static_cast<const int32_t*>(p.tokens)[row];
    const bool given = token >= 0 && token < p.vocab;
    Pass<T, WARPS> me(p, sh);
    me.c = p.inv_temperature * kLog2e;
    me.tok = given ? (int)token : p.vocab;
    me.xt = given ? Vec<T>::one(x + me.tok) : INFINITY;
    me.nan_token = me.xt != me.xt;
    me.c2 = two(me.c, me.c);
    me.base2 = 0;
    me.limit = -INFINITY;
    me.s2 = me.w2 = 0;
    me.ahead = 0;
    me.largest = me.bound = me.least = -INFINITY;
    me.own = 0;
    me.waiting = 0;
    const int share = TOP ? (p.top + WARPS - 1) / WARPS : 1;
    if (TOP) {
        // The CTA's bound from its first vectors: `share` lanes of every warp have an entry as large.
        float f[8];
        u0.get(f);
        me.largest = max8(f);
        u1.get(f);
        me.largest = fmaxf(fmaxf(me.largest, max8(f)), -INFINITY);
        __syncthreads();
        me.mark(share);
        __syncthreads();
        me.renew();
    }
#pragma unroll 1
    for (int it = 1; at - tid < v1; at += 2 * kThreads, ++it) {
        const Vec<T> c0 = u0, c1 = u1;
        load(at + 2 * kThreads);
        float f[8];
        c0.get(f);
        const float vm0 = max8(f);
        me.sum(f, vm0);
        me.count(f, vm0, head + 8 * at, at < v1 ? 0xffu : 0u);
        c1.get(f);
        const float vm1 = max8(f);
        me.sum(f, vm1);
        me.count(f, vm1, head + 8 * (at + kThreads), at + kThreads < v1 ? 0xffu : 0u);
        if (TOP) {
            const float vm = fmaxf(vm0, vm1);
            me.largest = fmaxf(me.largest, vm);
            if (me.wanted(vm0) && at < v1) me.push(vm0, at + 1);
            if (me.wanted(vm1) && at + kThreads < v1) me.push(vm1, at + kThreads + 1);
            // (at once where most lanes' first are wanted, as in a row that is masked but for a few)
            if ((it & 3) == 0 ? __any_sync(kAll, me.waiting > kSettle) : it == 1 && __popc(__ballot_sync(kAll, me.waiting > 1)) > 16) me.thin();
            if ((it & (it - 1)) == 0 && it > 1) {
                me.mark(share);
                __syncwarp();
                me.renew();
            }
        }
    }
    // The head and the tail, as vectors 0 and n_vec + 1: two lanes of the first part's first warp.
    if (part == 0 && warp == 0) {
        const int i0 = lane == 0 ? 0 : tail, n = lane == 0 ? head : lane == 1 ? p.vocab - tail : 0;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = k < n ? Vec<T>::one(x + i0 + k) : -INFINITY;
        me.sum(f, max8(f));
        float vm = f[0];                                       // (of entries that are there: a NaN is less than -inf)
#pragma unroll
        for (int k = 1; k < 8; ++k) vm = k < n ? fmaxf(vm, f[k]) : vm;
        if (n) me.count(f, vm, i0, (1u << n) - 1);
        if (TOP && n) me.push(vm, lane == 0 ? 0 : n_vec + 1);
    }

    // the warp's sums, then the block's, then the cluster's
    Sums a = me.sums();
    int ahead = me.ahead;
    auto reduce = [&](int lanes) {
#pragma unroll 1
        for (int o = lanes >> 1; o; o >>= 1) {
            const Sums b = {__shfl_xor_sync(kAll, a.m, o), __shfl_xor_sync(kAll, a.s, o), __shfl_xor_sync(kAll, a.w, o)};
            // (the lower lane's first in both, so that both have the same bits)
            const bool upper = lane & o;
            a = join(upper ? b : a, upper ? a : b, me.c);
            ahead += __shfl_xor_sync(kAll, ahead, o);
        }
    };
    reduce(32);
    if (lane == 0) sh.part[warp] = Part{a, ahead};
    if (TOP) {
        // the warp's last bound, and what it leaves of the entries that wait, at most 32 of a warp, to the pool
        me.mark(share);
        __syncthreads();
        me.renew();
        const uint64_t floor = (uint64_t)(me.bound == -INFINITY ? 0 : ordered(me.bound)) << 32;
        uint64_t* mine = sh.pending[warp];
        const int left = me.settled() & 63;
        int place = 0;
        if (lane == 0) place = atomicAdd(&sh.pooled, left);
        place = __shfl_sync(kAll, place, 0);
        if (lane < left) sh.pool[place + lane] = ordered_key(mine[lane]);
        choose(sh, p.top);
        __syncthreads();
        // the vectors' entries
        uint64_t key[8 / WARPS];
        for (int j = 0; j < 8 / WARPS; ++j) key[j] = sh.list[j * (kThreads / 8) + (tid >> 3)];
        clear(sh);
#pragma unroll
        for (int j = 0; j < 8 / WARPS; ++j) {
            const int vector = key_index(key[j]), entry = (vector ? head + 8 * (vector - 1) : 0) + (tid & 7);
            const bool on = key[j] && entry < (vector ? p.vocab : head);     // (the list has `top` keys)
            const uint64_t found = on ? key_of(Vec<T>::one(x + entry), entry) : 0;
            bring(sh, found >= floor ? found : 0);
        }
        choose(sh, p.top);
    }
    __syncthreads();
    auto take = [&](int n) {                                   // the first n parts', every lane the same
        a = sh.part[lane & (n - 1)].sums;
        ahead = sh.part[lane & (n - 1)].ahead;
        reduce(n);
    };
    if (warp == 0) take(WARPS);
    if (WARPS == 8 && parts > 1) {
        if (tid == 0) sh.cta_part = Part{a, ahead};
        dev::cluster_sync();
        if (part == 0) {
            // warp w takes part w's
            uint64_t key = 0;
            Part b = {{-INFINITY, 0.f, 0.f}, 0};
            if (warp < parts) {
                const uint32_t pa = dev::map_to_rank(dev::smem_addr(&sh.cta_part), (uint32_t)warp);
                if (TOP)
                    asm volatile("ld.shared::cluster.u64 %0, [%1];"
                                 : "=l"(key)
                                 : "r"(dev::map_to_rank(dev::smem_addr(&sh.list[lane]), (uint32_t)warp))
                                 : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.sums.m) : "r"(pa) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1+4];" : "=f"(b.sums.s) : "r"(pa) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1+8];" : "=f"(b.sums.w) : "r"(pa) : "memory");
                asm volatile("ld.shared::cluster.u32 %0, [%1+12];" : "=r"(b.ahead) : "r"(pa) : "memory");
            }
            if (lane == 0) sh.part[warp] = b;
            if (TOP) {
                // no key behind some part's top-th is among the first
                const uint64_t last = (uint64_t)__shfl_sync(kAll, (uint32_t)(key >> 32), p.top - 1) << 32 | __shfl_sync(kAll, (uint32_t)key, p.top - 1);
                if (lane == 0) sh.pending[0][warp] = last;
                __syncthreads();
                uint64_t floor = 0;
                for (int i = 0; i < parts; ++i) floor = max(floor, sh.pending[0][i]);
                clear(sh);
                cluster_arrive();                              // (the parts have been read)
                bring(sh, lane < p.top && key >= floor ? key : 0);
                choose(sh, p.top);
            } else {
                __syncthreads();
                cluster_arrive();
            }
            if (warp == 0) take(parts);
            __syncthreads();
        } else {
            cluster_arrive();
        }
    }
    if (part != 0 || warp != 0) {
        if (WARPS == 8 && parts > 1) cluster_wait();           // until the first part has read this one's
        return;
    }
    const float log_s = logf(a.s);                             // (a row of -inf alone: log 0)
    auto lp = [&](float v) { return v == -INFINITY && a.s == a.s ? v : (v - from(a.m)) * p.inv_temperature - log_s; };
    if (lane == 0) {
        if (p.entropy) p.entropy[row] = a.s == 0.f ? 0.f : log_s - kLn2 * (a.w / a.s);
        if (p.logprobs) p.logprobs[row] = given ? lp(me.xt) : __uint_as_float(0x7fc00000u);
        if (p.ranks) p.ranks[row] = given ? ahead : -1;
    }
    if (TOP && lane < p.top) {
        const uint64_t key = sh.list[lane];
        p.top_logprobs[row * p.top + lane] = lp(key_value(key));
        p.top_tokens[row * p.top + lane] = key_index(key);
    }
    __syncwarp();
    if (WARPS == 8 && parts > 1) cluster_wait();
}

}  // namespace

cudaError_t launch_token_logprobs(const ScoreParams& p, cudaStream_t stream) {
    // A cluster a row while rows are few: half of the GPU's room for blocks (four an SM) filled, and parts of at least
    // 2,048 entries.
    int parts = 1;
    while (parts < 8 && (long long)p.rows * parts * 2 <= 608 && p.vocab / (parts * 2) >= 2048) parts *= 2;
    // Blocks of four warps, eight an SM, where rows are many or short: a row's last choice leaves half as many lanes idle.
    // With 20 alternatives, eight warps and four: 4,096 rows of 100,003 227 and 213 us, 2,048 121 and 120, 1,300 84 and 90,
    // 1,300 of 10,003 27 and 22, 700 18 and 16, 8,192 of 4,000 101 and 68.
    const bool small = parts == 1 && (p.rows >= 2048 || (p.rows > 608 && p.vocab <= 32768));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)parts, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows * parts);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto go = [&](auto eight, auto four) {
        cfg.blockDim = dim3(small ? 128 : 256);
        return cudaLaunchKernelEx(&cfg, small ? four : eight, p);
    };
    if (p.top)
        return p.is_fp32 ? go(token_logprobs_kernel<float, true, 8>, token_logprobs_kernel<float, true, 4>)
                         : go(token_logprobs_kernel<__nv_bfloat16, true, 8>, token_logprobs_kernel<__nv_bfloat16, true, 4>);
    return p.is_fp32 ? go(token_logprobs_kernel<float, false, 8>, token_logprobs_kernel<float, false, 4>)
                     : go(token_logprobs_kernel<__nv_bfloat16, false, 8>, token_logprobs_kernel<__nv_bfloat16, false, 4>);
}

}  // namespace lora
