// What stands before an 8-bit projection: the gated activation between gate_up and down (bf16 or 8-bit output), rows
// and weights brought to 8 bits. Each reads its input once and is bound by memory (on a few rows by one pass's latency).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dev_common.cuh"
#include "layer_internal.h"

namespace lora {
namespace {

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(dev::pack_bf16x2(f[0], f[1]), dev::pack_bf16x2(f[2], f[3]), dev::pack_bf16x2(f[4], f[5]),
                      dev::pack_bf16x2(f[6], f[7]));
}
// max that keeps a NaN of either side, so that a group with one gets a NaN scale
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax8(const float* f) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max_nan(m, fabsf(f[k]));
    return m;
}
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) {   // of two bf16's magnitudes each; keeps a NaN
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
    return r;
}
// scale of a maximum, floored so that its reciprocal is finite and zeros are exact (as the norm's in 8 bits)
__device__ __forceinline__ float scale_of(float amax) {
    const float s = amax * (1.0f / 448.f);
    return s < 7.888609052210118e-31f ? 7.888609052210118e-31f : s;   // 2^-100; a NaN stays
}
__device__ __forceinline__ uint2 to_e4m3(const float* f, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float exp2_of(float t) {      // 2^-22 of the value; 0 below 2^-126
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}
// g / (1 + e^-g) u as (g / 4) (1 / (1/4 + e^-g / 4)) u: the reciprocal is no subnormal however large e^-g is (__fdividef is 0
// from 2^126 on). e^-g itself is infinite from g = -88.7 on, where a large u still gives a y that is not 0: gates below -80,
// which are rare, take g h u h with h = e^(g / 2) (1 + h^2 is 1), 0 only where no bf16 y is left; threads without one do not
// ask (FAR). (g u / (1 + h^2) with h = e^(-|g| / 2), times h twice below 0, for all gates: 4,001 rows of 17,408 to 8 bits
// 69 us by groups, 90 by rows.)
template <bool FAR>
__device__ __forceinline__ void silu_mul8(const uint4& gate, const uint4& up, float* y) {
    constexpr float kLog2e = 1.4426950408889634f;
    float u[8];
    unpack8(gate, y);
    unpack8(up, u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float g = y[k];
        float r, h;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(exp2_of(g * -kLog2e), 0.25f, 0.25f)));
        y[k] = 0.25f * g * r * u[k];
        if (FAR && g < -80.f) {
            asm("ex2.approx.f32 %0, %1;" : "=f"(h) : "f"(g * (0.5f * kLog2e)));              // (subnormal from g = -174 on)
            y[k] = g * h * u[k] * h;
        }
    }
}
// Whether a thread's gates go below -80.
template <int N>
__device__ __forceinline__ bool far_gates(const uint4 (&a)[N]) {
    uint32_t m = a[0].x;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (const uint32_t w : {a[i].x, a[i].y, a[i].z, a[i].w}) asm("min.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
    return fminf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u)) < -80.f;
}

// One row's vector c (8 features) of the operator's values in fp32.
template <bool GATE, bool FAR>
__device__ __forceinline__ void values8(const uint4& a, const uint4& b, float* y) {
    if (GATE) silu_mul8<FAR>(a, b, y);
    else unpack8(a, y);
}

// Scales by groups, or bf16 alone: a warp takes pieces of 32 vectors of a row (256 features, whole groups), one where
// there are few and N beside one another, all in flight, where there are many. No loop: as blocks end others begin, so
// that loads and stores of an SM overlap (blocks that stayed and looped over their pieces: 4,001 rows of 17,408 to bf16
// 67.2 us for 60.6, 1,601 rows of 5,120 to 8 bits 7.9 for 6.4). To bf16 bound by memory (4,001 rows: 6.9 TB/s), to 8 bits
// by instructions beside it (5.1 to 5.5 TB/s).
template <bool GATE, int N, int B>
__global__ void __launch_bounds__(256, B) act_groups_kernel(const __grid_constant__ ActParams p) {
    dev::griddep_wait();
    dev::griddep_launch_dependents();
    const int nvec = p.width >> 3, per_row = (nvec + 31) >> 5, lane = threadIdx.x & 31;
    const int lanes = p.group >> 3, shift = p.group ? 31 - __clz(lanes) : 0, ng = p.group ? (nvec + lanes - 1) >> shift : 0;
    const long long first = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * N;
    int row = first < (1ll << 31) ? (int)((uint32_t)first / (uint32_t)per_row) : (int)(first / per_row), at = (int)(first - (long long)row * per_row);
    uint4 a[N], b[N];
    int rows[N], c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        rows[i] = row;
        c[i] = row < p.rows ? at * 32 + lane : nvec;
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        if (c[i] < nvec) {
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + row * p.x_stride;
            a[i] = __ldcs(reinterpret_cast<const uint4*>(x) + c[i]);
            if (GATE) b[i] = __ldcs(reinterpret_cast<const uint4*>(x + p.width) + c[i]);
        }
        if (++at == per_row) {
            at = 0;
            ++row;
        }
    }
    const bool far = GATE && far_gates(a);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (rows[i] >= p.rows) break;
        float y[8];
        if (far) values8<GATE, true>(a[i], b[i], y);
        else values8<GATE, false>(a[i], b[i], y);
        if (p.y && c[i] < nvec) reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + rows[i] * p.y_stride)[c[i]] = pack8(y);
        if (!p.q8) continue;
        float m;
        if (GATE) {
            m = amax8(y);
        } else {                                           // (exact in bf16)
            const uint32_t m2 = amax2(amax2(amax2(a[i].x & 0x7fff7fffu, a[i].y), a[i].z), a[i].w);
            m = max_nan(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
        }
        for (int o = lanes >> 1; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (c[i] < nvec) {
            const float s = scale_of(m);
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q8) + rows[i] * p.q8_stride)[c[i]] = to_e4m3(y, __frcp_rn(s));
            if ((c[i] & (lanes - 1)) == 0) p.scales[(long long)rows[i] * ng + (c[i] >> shift)] = s;
        }
    }
}

// One scale a row: a block a row, which stays in registers between its maximum and its output (4,001 rows of 17,408 gated
// 52 us, 6.7 TB/s; 48 rows 3.0). Registers for two blocks an SM: 17,408 features are 544 threads, at 64 registers one block
// and 76 us; 12,288 are 768, at 48 one block and 78 us for 55 (5,668 rows).
template <bool GATE, int V>
__global__ void __maxnreg__(V == 1 ? 32 : V == 2 ? 40 : 56) act_rows_kernel(const __grid_constant__ ActParams p) {
    __shared__ float buf[32];
    dev::griddep_wait();
    dev::griddep_launch_dependents();
    const long long row = blockIdx.x;
    const int nvec = p.width >> 3, tid = threadIdx.x, nt = blockDim.x;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + row * p.x_stride;
    uint4 a[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        if (c < nvec) {
            a[i] = reinterpret_cast<const uint4*>(x)[c];
            if (GATE) b[i] = reinterpret_cast<const uint4*>(x + p.width)[c];
        }
    }
    float y[V][8], m = 0.f;
    if (GATE && far_gates(a)) {
#pragma unroll
        for (int i = 0; i < V; ++i) values8<GATE, true>(a[i], b[i], y[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) values8<GATE, false>(a[i], b[i], y[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) m = max_nan(m, amax8(y[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) buf[tid >> 5] = m;
    __syncthreads();
    m = (tid & 31) < (nt >> 5) ? buf[tid & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = scale_of(m), inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        if (c >= nvec) continue;
        if (p.y) reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + row * p.y_stride)[c] = pack8(y[i]);
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q8) + row * p.q8_stride)[c] = to_e4m3(y[i], inv);
    }
    if (tid == 0) p.scales[row] = s;
}

// A weight's block of 128 x 128: 256 threads hold it, eight vectors each, between its maximum and its output; four blocks an
// SM. Bound by memory: 34,816 x 5,120 in 77.5 us, 6.9 TB/s. (With the maximum taken of unpacked values, 88 registers a
// thread and two blocks an SM, 95.7; 512 threads of four vectors 81.4; five blocks, which spill, 86.7.)
__global__ void __launch_bounds__(256, 4) fp8_blocks_kernel(const __grid_constant__ BlocksParams p) {
    constexpr int V = 8, kWarps = 64 / V, kRows = 128 / V;   // rows apart of a thread's vectors
    __shared__ float buf[kWarps];
    dev::griddep_wait();
    dev::griddep_launch_dependents();
    const int nc = (p.cols + 127) >> 7, br = (int)(blockIdx.x / nc), bc = (int)(blockIdx.x % nc);
    const int col = bc * 128 + (threadIdx.x & 15) * 8, r0 = br * 128 + (threadIdx.x >> 4);
    uint4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int r = r0 + kRows * i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < p.rows && col < p.cols)
            v[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.w) + (long long)r * p.w_stride + col));
    }
    uint32_t m2 = 0;                                       // two features' maxima (exact in bf16)
#pragma unroll
    for (int i = 0; i < V; ++i) m2 = amax2(amax2(amax2(amax2(m2, v[i].x), v[i].y), v[i].z), v[i].w);
    float m = max_nan(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = m;
    __syncthreads();
    m = buf[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = scale_of(m), inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int r = r0 + kRows * i;
        if (r >= p.rows || col >= p.cols) continue;
        float f[8];
        unpack8(v[i], f);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q8) + (long long)r * p.q8_stride + col) = to_e4m3(f, inv);
    }
    if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
}

template <bool GATE>
cudaError_t launch(const ActParams& p, cudaStream_t stream) {
    const int nvec = p.width >> 3;
    if (p.q8 && p.group == 0) {
        const int v = nvec > 2048 ? 4 : nvec > 1024 ? 2 : 1, nt = ((nvec + v - 1) / v + 31) / 32 * 32;
        if (v == 1) return launch_chained(act_rows_kernel<GATE, 1>, p.rows, nt, 0, stream, p);
        if (v == 2) return launch_chained(act_rows_kernel<GATE, 2>, p.rows, nt, 0, stream, p);
        return launch_chained(act_rows_kernel<GATE, 4>, p.rows, nt, 0, stream, p);
    }
    const long long pieces = (long long)p.rows * ((nvec + 31) / 32);
    auto go = [&](auto kernel, int n) { return launch_chained(kernel, (unsigned)((pieces + 8 * n - 1) / (8 * n)), 256, 0, stream, p); };
    // Pieces of a warp 1, 2 and 4, to 8 bits: 48 rows of 17,408 gated 2.2 us with one; 300 rows 7.2, 6.9, 8.0; 4,001 rows 71.7,
    // 67.1, 63.7; 600 rows of 5,120 as they are 3.4, 3.8, 3.4; 1,601 rows 7.3, 6.4, 6.7; 16,384 rows of 6,144 74.0, 58.4, 56.1.
    if (pieces <= 12000) return go(act_groups_kernel<GATE, 1, 8>, 1);
    if (pieces <= 65536) return go(act_groups_kernel<GATE, 2, 5>, 2);
    return go(act_groups_kernel<GATE, 4, 4>, 4);
}

}  // namespace

cudaError_t launch_act(const ActParams& p, bool gate, cudaStream_t stream) {
    return gate ? launch<true>(p, stream) : launch<false>(p, stream);
}

cudaError_t launch_fp8_blocks(const BlocksParams& p, cudaStream_t stream) {
    const long long blocks = (long long)((p.rows + 127) / 128) * ((p.cols + 127) / 128);
    return launch_chained(fp8_blocks_kernel, (unsigned)blocks, 256, 0, stream, p);
}

}  // namespace lora
