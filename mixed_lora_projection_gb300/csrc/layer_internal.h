// Internal declarations of the operators between the projections (include/lora_layer.h),
// shared by their translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lora {

constexpr int kMaxSeqs = 1024;          // sequences of one call: their row offsets travel in the kernel parameters
constexpr int kSmallSeqs = 64;          // calls of at most this many take 16 times smaller parameters

struct NormParams {
    const void* x;
    const void* residual;
    const void* weight;
    void* h;
    void* y;
    void* q8;
    float* scales;
    long long x_stride, r_stride, h_stride, y_stride, q8_stride;
    float weight_offset, eps;
    int rows, width, group;
};
cudaError_t launch_add_rms_norm(const NormParams& p, cudaStream_t stream);

// Where the tokens of the cached sequences are (lora_kv_cache).
struct CacheView {
    void* k;
    void* v;
    long long k_page, k_token, k_head;
    long long v_page, v_token, v_head;
    const int32_t* table;
    const int32_t* kv_lens;
    long long table_stride;
    int n_pages, page_size, n_kv, dim, pages_per_seq, n_seqs;
};

// Row offsets of the sequences: sequence i's new rows are [off[i], off[i + 1]).
template <int N>
struct SeqOffsets {
    int32_t off[N + 1];
};

struct AppendParams {
    CacheView c;
    const void* q;
    void* q_out;
    const void* k;
    const void* v;
    const float* cos;
    const float* sin;
    long long q_stride, q_head, qo_stride, qo_head, k_stride, k_head, v_stride, v_head;
    int n_heads, rot, n_positions, rows;
};
cudaError_t launch_kv_append(const AppendParams& p, const int32_t* q_offsets, cudaStream_t stream);

struct AttnParams {
    CacheView c;
    const void* q;
    void* out;
    long long q_stride, q_head, o_stride, o_head;
    int n_heads, rows, window, sinks;
    float scale_log2;                   // softmax in base 2: scale * log2(e)
    int* status;
    unsigned long long wait_limit_ns;
};

cudaError_t launch_attention(const AttnParams& p, const int32_t* q_offsets, cudaStream_t stream);

}  // namespace lora
