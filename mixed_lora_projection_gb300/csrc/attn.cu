// Attention of a batch's new rows over the paged cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "layer_internal.h"

namespace lora {
namespace {

// One warp per (row, head): 32 keys at a time, one per lane, with the running maximum and sum;
// each lane then adds the 32 values' share of D / 32 features.
template <int D, int N>
__global__ void __launch_bounds__(128) attn_kernel(const __grid_constant__ AttnParams p,
                                                   const __grid_constant__ SeqOffsets<N> o) {
    constexpr int E = D / 32;
    typedef __nv_bfloat16 bf;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 4 + warp;
    if (item >= (long long)p.rows * p.n_heads) return;
    const int t = (int)(item / p.n_heads), head = (int)(item % p.n_heads);
    const int kh = head / (p.n_heads / p.c.n_kv);
    int lo = 0, hi = p.c.n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (o.off[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const long long cap = (long long)p.c.pages_per_seq * p.c.page_size;
    const int len = (int)min((long long)max(p.c.kv_lens[lo], 0), cap);
    const int pos = len - (o.off[lo + 1] - t);
    const bf* q = static_cast<const bf*>(p.q) + t * p.q_stride + head * p.q_head;
    for (int i = lane; i < D; i += 32) qs[warp][i] = __bfloat162float(q[i]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[E];
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const int first = p.window ? max(0, pos - p.window + 1) : 0;
    const int sinks = min(p.sinks, first);
    // chunks over the sinks, then over the window
    for (int part = 0; part < 2; ++part) {
        const int a = part ? first : 0, b = part ? pos + 1 : sinks;
        for (int j0 = a; j0 < b; j0 += 32) {
            const int j = j0 + lane;
            float s = -INFINITY;
            int page = -1;
            if (j < b) {
                page = p.c.table[lo * p.c.table_stride + j / p.c.page_size];
                if (page < 0 || page >= p.c.n_pages) page = -1;
                s = 0.f;
                if (page >= 0) {
                    const bf* k = static_cast<const bf*>(p.c.k) + page * p.c.k_page +
                                  (j % p.c.page_size) * p.c.k_token + kh * p.c.k_head;
                    for (int i = 0; i < D; ++i) s = fmaf(qs[warp][i], __bfloat162float(k[i]), s);
                }
                s *= p.scale_log2;
            }
            float mx = s;
            for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
            const float alpha = exp2f(m - ms), w = exp2f(s - ms);
            m = mn;
            float sum = w;
            for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l = l * alpha + sum;
            for (int e = 0; e < E; ++e) acc[e] *= alpha;
            for (int i = 0; i < 32 && j0 + i < b; ++i) {
                const float pi = __shfl_sync(0xffffffffu, w, i);
                const int pg = __shfl_sync(0xffffffffu, page, i);
                if (pg < 0) continue;
                const bf* v = static_cast<const bf*>(p.c.v) + pg * p.c.v_page +
                              ((j0 + i) % p.c.page_size) * p.c.v_token + kh * p.c.v_head;
                for (int e = 0; e < E; ++e) acc[e] = fmaf(pi, __bfloat162float(v[lane + 32 * e]), acc[e]);
            }
        }
    }
    bf* out = static_cast<bf*>(p.out) + t * p.o_stride + head * p.o_head;
    for (int e = 0; e < E; ++e) out[lane + 32 * e] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[e] / l);
}

template <int D, int N>
cudaError_t launch(const AttnParams& p, const int32_t* off, cudaStream_t stream) {
    SeqOffsets<N> o;
    for (int i = 0; i <= p.c.n_seqs; ++i) o.off[i] = off[i];
    const long long items = (long long)p.rows * p.n_heads;
    attn_kernel<D, N><<<(unsigned)((items + 3) / 4), 128, 0, stream>>>(p, o);
    return cudaGetLastError();
}

template <int N>
cudaError_t by_dim(const AttnParams& p, const int32_t* off, cudaStream_t stream) {
    if (p.c.dim == 64) return launch<64, N>(p, off, stream);
    if (p.c.dim == 128) return launch<128, N>(p, off, stream);
    return launch<256, N>(p, off, stream);
}

}  // namespace

cudaError_t launch_attention(const AttnParams& p, const int32_t* q_offsets, cudaStream_t stream) {
    return p.c.n_seqs <= kSmallSeqs ? by_dim<kSmallSeqs>(p, q_offsets, stream) : by_dim<kMaxSeqs>(p, q_offsets, stream);
}

}  // namespace lora
