// The residual's addition with the root-mean-square norm (bf16 or 8-bit output), and the append
// of new keys and values to the paged cache with the rotary turn. Both move each byte once and
// are bound by memory (or, on a few rows, by the latency of one pass).
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
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// max that keeps a NaN of either side, so that a row with one gets NaN scales
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Reduces v over the block (NT threads) or, in the warp form, over the warp; every thread gets it.
template <bool WARP, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_nan(v, w) : v + w;
    }
    if (WARP) return v;
    const int n = (int)(blockDim.x >> 5), lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < n ? buf[lane] : 0.f;      // sums of squares and magnitudes: 0 is neutral to both
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_nan(v, w) : v + w;
    }
    return v;
}

constexpr float kE4m3Max = 448.f;

// 8-bit output: scale of a maximum, floored so that its reciprocal is finite and a zero row is exact.
__device__ __forceinline__ float scale_of(float amax) {
    const float s = amax * (1.0f / kE4m3Max);
    return s < 7.888609052210118e-31f ? 7.888609052210118e-31f : s;   // 2^-100; a NaN stays
}

__device__ __forceinline__ uint2 to_e4m3(const float* f, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi =
            __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    return make_uint2(w[0], w[1]);
}

// h = x + residual, y = h (mean h^2 + eps)^(-1/2) (weight + offset); 8 bits: s = max(max|y| / 448, 2^-100),
// q = e4m3(y / s). One row per block (or per warp: WARP), V 16-byte vectors of it per thread. The row stays
// in registers (fp32) between its sum of squares and its outputs, so x and the residual are read once and
// memory is the bound: 16,384 rows of 5,120 with a residual take 100 us in bf16 (0.99 of the measured copy
// rate) and 87-90 us to 8 bits (0.96-1.0); 48 rows take one pass's latency, 1.8 us back to back in a graph. The weights are read after the
// sum, when the sum's loads have left their registers (4,096 rows of 17,408: 82 us against 125).
template <int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) add_rms_norm_kernel(const NormParams p) {
    __shared__ float buf[2][32];
    const int nt = WARP ? 32 : (int)blockDim.x;
    const int tid = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int row = WARP ? (int)(blockIdx.x * 4 + (threadIdx.x >> 5)) : (int)blockIdx.x;
    dev::griddep_wait();
    dev::griddep_launch_dependents();
    if (WARP && row >= p.rows) return;
    const int nvec = p.width >> 3;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + row * p.x_stride);
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.residual) + row * p.r_stride);
    const uint4* w = static_cast<const uint4*>(p.weight);
    uint4 xv[V], rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        const uint4 z = make_uint4(0, 0, 0, 0);
        xv[i] = c < nvec ? x[c] : z;
        rv[i] = (p.residual && c < nvec) ? r[c] : z;
    }
    float h[V][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float b[8];
        unpack8(xv[i], h[i]);
        if (p.residual) {
            unpack8(rv[i], b);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] += b[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(h[i][k], h[i][k], ss);
    }
    if (p.h) {
        uint4* ho = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.h) + row * p.h_stride);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tid + i * nt < nvec) ho[tid + i * nt] = pack8(h[i]);
    }
    ss = row_reduce<WARP, false>(ss, buf[0]);
    const float inv = rsqrtf(ss / (float)p.width + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float b[8];
        unpack8(tid + i * nt < nvec ? w[tid + i * nt] : make_uint4(0, 0, 0, 0), b);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] = h[i][k] * inv * (b[k] + p.weight_offset);
    }
    if (p.y) {
        uint4* yo = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + row * p.y_stride);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tid + i * nt < nvec) yo[tid + i * nt] = pack8(h[i]);
    }
    if (!p.q8) return;
    uint2* qo = reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q8) + row * p.q8_stride);
    float amax[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        amax[i] = 0.f;
        // a thread past the row's end holds zeros (0 * inv), unless inv is not finite
#pragma unroll
        for (int k = 0; k < 8; ++k) amax[i] = max_nan(amax[i], fabsf(h[i][k]));
        if (tid + i * nt >= nvec) amax[i] = 0.f;
    }
    if (p.group == 0) {
        float m = amax[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = max_nan(m, amax[i]);
        const float s = scale_of(row_reduce<WARP, true>(m, buf[1]));
        const float si = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tid + i * nt < nvec) qo[tid + i * nt] = to_e4m3(h[i], si);
        if (tid == 0) p.scales[row] = s;
        return;
    }
    // a group is group / 8 vectors: as many neighbouring lanes, since nt is a multiple of 32
    const int lanes = p.group >> 3, shift = 31 - __clz(lanes), ng = (nvec + lanes - 1) >> shift;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        float m = amax[i];
        for (int o = lanes >> 1; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = scale_of(m);
        if (c < nvec) {
            qo[c] = to_e4m3(h[i], __frcp_rn(s));
            if ((c & (lanes - 1)) == 0) p.scales[(long long)row * ng + (c >> shift)] = s;
        }
    }
}

// Turns 8 features of each half: (a, b) -> (a cos - b sin, b cos + a sin).
__device__ __forceinline__ void turn8(float* a, float* b, const float* cs, const float* sn) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 c4 = *reinterpret_cast<const float4*>(cs + i), s4 = *reinterpret_cast<const float4*>(sn + i);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = a[i + k], y = b[i + k];
            a[i + k] = x * c[k] - y * s[k];
            b[i + k] = y * c[k] + x * s[k];
        }
    }
}

// One block per new row: its sequence, position and place in the cache once, then its heads' 16-byte
// vectors, those of the two rotary halves in pairs. Bound by memory: 16,384 rows of 24 + 2 x 12 heads of
// 256 take 129-133 us (0.89-0.92 of the measured copy rate) with 64 features turned, 129 with none.
template <int N>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendParams p,
                                                        const __grid_constant__ SeqOffsets<N> o) {
    const int t = blockIdx.x;
    int lo = 0, hi = p.c.n_seqs - 1;                 // the last sequence that begins at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (o.off[mid] <= t) lo = mid; else hi = mid - 1;
    }
    dev::griddep_wait();
    dev::griddep_launch_dependents();
    const long long cap = (long long)p.c.pages_per_seq * p.c.page_size;
    const int len = (int)min((long long)max(p.c.kv_lens[lo], 0), cap);
    const int pos = len - (o.off[lo + 1] - t);
    const int rp = min(max(pos, 0), p.n_positions - 1);
    int page = -1, slot = 0;
    if (pos >= 0) {
        page = p.c.table[lo * p.c.table_stride + pos / p.c.page_size];
        slot = pos % p.c.page_size;
        if (page >= p.c.n_pages) page = -1;
    }
    // items of 16 bytes: pairs of the two rotary halves (two of them each), the turned heads' other features,
    // the values; kinds one after another, so that few warps have two of them
    const int pairs = p.rot >> 4, single = (p.c.dim - p.rot) >> 3, per_v = p.c.dim >> 3;
    const int nq = p.q_out ? p.n_heads : 0, heads = nq + (page >= 0 ? p.c.n_kv : 0);
    const int n_pairs = heads * pairs, n_turned = n_pairs + heads * single, end = n_turned + (page >= 0 ? p.c.n_kv * per_v : 0);
    const float* cs = p.cos + (long long)rp * (p.rot >> 1);
    const float* sn = p.sin + (long long)rp * (p.rot >> 1);
    typedef __nv_bfloat16 bf;
    bf* kd = static_cast<bf*>(p.c.k) + page * p.c.k_page + slot * p.c.k_token;
    bf* vd = static_cast<bf*>(p.c.v) + page * p.c.v_page + slot * p.c.v_token;
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < end; i += gridDim.y * blockDim.x) {
        if (i >= n_turned) {
            const int u = i - n_turned, h = u / per_v, c = u - h * per_v;
            const bf* s = static_cast<const bf*>(p.v) + t * p.v_stride + h * p.v_head;
            reinterpret_cast<uint4*>(vd + h * p.c.v_head)[c] = reinterpret_cast<const uint4*>(s)[c];
            continue;
        }
        const bool pair = i < n_pairs;
        const int per = pair ? pairs : single, u = pair ? i : i - n_pairs, hh = u / per, c = u - hh * per;
        const bool is_q = hh < nq;
        const int h = is_q ? hh : hh - nq;
        const bf* s = is_q ? static_cast<const bf*>(p.q) + t * p.q_stride + h * p.q_head
                           : static_cast<const bf*>(p.k) + t * p.k_stride + h * p.k_head;
        bf* d = is_q ? static_cast<bf*>(p.q_out) + t * p.qo_stride + h * p.qo_head : kd + h * p.c.k_head;
        if (!pair) {
            const int e = p.rot + (c << 3);
            *reinterpret_cast<uint4*>(d + e) = *reinterpret_cast<const uint4*>(s + e);
            continue;
        }
        const int e = c << 3, f = e + (p.rot >> 1);
        float a[8], b[8];
        unpack8(*reinterpret_cast<const uint4*>(s + e), a);
        unpack8(*reinterpret_cast<const uint4*>(s + f), b);
        turn8(a, b, cs + e, sn + e);
        *reinterpret_cast<uint4*>(d + e) = pack8(a);
        *reinterpret_cast<uint4*>(d + f) = pack8(b);
    }
}

}  // namespace

cudaError_t launch_add_rms_norm(const NormParams& p, cudaStream_t stream) {
    const int nvec = p.width >> 3;
    if (nvec <= 128) {
        const int grid = p.rows / 4 + (p.rows % 4 != 0);
        if (nvec <= 32) return launch_chained(add_rms_norm_kernel<1, true>, grid, 128, 0, stream, p);
        if (nvec <= 64) return launch_chained(add_rms_norm_kernel<2, true>, grid, 128, 0, stream, p);
        return launch_chained(add_rms_norm_kernel<4, true>, grid, 128, 0, stream, p);
    }
    // Vectors a thread. On few rows the latency counts: 48 rows of 5,120 back to back 1.8 us with one against 2.1 with
    // four, 304 rows of 12,288 3.8 with two against 4.8. On many, the rows in flight: 1,601 rows of 5,120 6.6 us with
    // four against 8.2 with one, of 16,384 from HBM 37 with four against 43 with two. Around 304 rows (two blocks an SM)
    // it goes either way: 304 of 5,120 2.9 with one against 2.6, 608 4.2 against 4.5 with four.
    const int v = nvec > 2048 || p.rows > 304 ? 4 : nvec > 1024 ? 2 : 1;
    const int nt = ((nvec + v - 1) / v + 31) / 32 * 32;
    if (v == 1) return launch_chained(add_rms_norm_kernel<1, false>, p.rows, nt, 0, stream, p);
    if (v == 2) return launch_chained(add_rms_norm_kernel<2, false>, p.rows, nt, 0, stream, p);
    return launch_chained(add_rms_norm_kernel<4, false>, p.rows, nt, 0, stream, p);
}

template <int N>
static cudaError_t append(const AppendParams& p, const int32_t* off, cudaStream_t stream) {
    SeqOffsets<N> o;
    for (int i = 0; i <= p.c.n_seqs; ++i) o.off[i] = off[i];
    // A few rows are shared out to several blocks each, one vector a thread (at most two blocks an SM): 48 rows of
    // 24 + 2 x 12 heads of 256 take 2.2 us in a graph (3.9 with a block a row, before the kernels' order of
    // waiting changed; 2.6 with several then).
    const long long items = (long long)((p.q_out ? p.n_heads : 0) + 2 * p.c.n_kv) * (p.c.dim >> 3);
    const unsigned per_row = (unsigned)std::max(1ll, std::min((items + 255) / 256, 304ll / p.rows));
    return launch_chained(kv_append_kernel<N>, dim3(p.rows, per_row), 256, 0, stream, p, o);
}

cudaError_t launch_kv_append(const AppendParams& p, const int32_t* q_offsets, cudaStream_t stream) {
    return p.c.n_seqs <= kSmallSeqs ? append<kSmallSeqs>(p, q_offsets, stream) : append<kMaxSeqs>(p, q_offsets, stream);
}

}  // namespace lora
