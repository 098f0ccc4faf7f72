// Internal declarations of the operators between the projections (include/lora_layer.h),
// shared by their translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lora {

// Launches a kernel that may begin while the stream's kernel before it ends: its blocks wait for that kernel
// (griddep_wait) before they read or write global memory, and only then let the next one begin
// (griddep_launch_dependents), which may read what it takes for finished before it waits itself (LORA_OPT_PDL: W).
// Steps of decode are chains of kernels of a few microseconds, where the launches' latency counts: back to back in a
// graph, the norm of 48 rows takes 1.8 us (4.1 with ordinary launches), the append of 48 rows 2.2 (6.2); letting the
// next one begin before the wait, which is not safe, 1.8 and 3.1.
template <class... Params, class... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

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

constexpr int kNoStall = 1 << 30;       // more tiles than a unit has

struct AttnParams {
    CacheView c;
    const void* q;
    void* out;
    long long q_stride, q_head, o_stride, o_head;
    int n_heads, rows, window, sinks;
    float scale_log2;                   // softmax in base 2: scale * log2(e)
    int* status;
    unsigned long long wait_limit_ns;
    int debug_stall;                    // n > 0: a load warp stops after n - 1 tiles of K and V (tests)
    cudaStream_t stream;
};

// The sequences one launch works on: their index in the call, first row and number of rows.
template <int N>
struct SeqList {
    int32_t n;
    int32_t row[N];
    int32_t q_len[N];
    uint16_t seq[N];
};

constexpr int kDecodeRows = 16;         // most rows per key/value head of a sequence in the decode kernel

struct DecodeParams {
    CUtensorMap tm_k, tm_v;             // box: 64 features of one head x granule tokens of one page
    AttnParams a;
    int k_order, v_order;               // order of the maps' axes (dev::tma_load_kv)
    int granule;                        // tokens of one load: divides the page size and the tile
    int group;                          // query heads per key/value head
    int slots;                          // ring slots of one tile of K or V
    float* part_o;                      // [2 x grid][16][dim]: unnormalised sums of split units
    float2* part_ml;                    // [2 x grid][16]: running maximum and sum
    uint32_t* prefix;                   // [n + 1]: tiles of one head before each sequence
    int most_rows;                      // of a sequence, per key/value head
    int grid;
};
size_t decode_smem(int dim, int slots, int seqs);
constexpr int kSmemTwo = 115200;        // the most dynamic shared memory that lets two blocks share an SM
cudaError_t decode_prepare_device();
cudaError_t launch_decode(const DecodeParams& p, const SeqList<kMaxSeqs>& seqs, cudaStream_t stream);

constexpr int kPromptBlocks = 152;      // most blocks of a launch, one per SM
constexpr int kPromptTile = 128;        // the prompt kernel's tile of rows and of cache tokens

// SeqList with the first unit of each sequence: a unit is one key/value head and the rows of
// PromptParams::tiles tiles.
template <int N>
struct PromptList : SeqList<N> {
    int32_t unit0[N];
};

struct PromptParams {
    CUtensorMap tm_k, tm_v;             // as DecodeParams
    CUtensorMap tm_q;                   // box: 64 features x the group's heads x tile_tokens tokens
    int q_outer;                        // the queries' heads are further apart than their tokens: a tile's rows then go
                                        // by head (row r is token r % tile_tokens), not by token (row r is head r % group)
    AttnParams a;
    int k_order, v_order, granule, group;
    int tile_tokens;                    // tokens of one tile of rows: 128 / group
    int tiles;                          // tiles of rows of a unit: 1 where no sequence needs more, else prompt_tiles(dim)
    int out32;                          // every row of the output is 32-byte aligned
    int join_rows;                      // rows of a unit that may hold a token
    int units, whole, blocks;           // units from `whole` on, fewer than blocks, may be cut in parts
    float* part_o;                      // [2 x blocks][tiles x 128][dim]: sums of units that parts end in
    float2* part_ml;
    uint32_t* prefix;                   // [kPromptBlocks + 2]: tiles before each of these, all of them, the longest's
    int* counter;                       // [2] units handed out past the first of each block; blocks that have ended
};
int prompt_tiles(int dim);              // most tiles of rows of a unit
cudaError_t prompt_prepare_device();
cudaError_t launch_prompt(const PromptParams& p, const PromptList<kMaxSeqs>& seqs, cudaStream_t stream);

}  // namespace lora
