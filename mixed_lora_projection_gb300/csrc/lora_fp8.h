// Internal declarations of the 8-bit-base kernel (kernels_fp8.cu) and its host side (not
// installed). Kept apart from lora_internal.h so that the other kernels' sources do not change
// when only this kernel's parameters do.
#pragma once

#include "lora_internal.h"

namespace lora {

constexpr int kFp8Group = 128;        // input features per scale; a base weight's block is 128 x 128
constexpr int kFp8Threads = 384;      // warp 0 TMA, 1 and 2 MMA, 3 scales (and owns TMEM), 4..11 epilogue
constexpr int kFp8MaxParts = 8;       // most parts of K: one CTA of a cluster each
constexpr int kFp8InlineAdapters = 8; // named in a call whose work list travels in the parameters
constexpr int kFp8Expands = 16;       // pairs of a row tile and an adapter, where tiles hold several
constexpr int kFp8StageRow = 128;     // bytes of a stage's row: one group of e4m3, 64 bf16 of the expand

// In place of a tile's split_index: a tile without an adapter that shares an SM pair, and so the expand, with an adapter's.
// Its rows take nothing of the expand (its U is zeros, but zero times a NaN of the adapter's is none).
constexpr int kApart = -1;

// One expand of a tile that holds rows of several adapters.
struct Fp8Expand {
    int adapter, slot;                // its U is the 128 rows from 128 slot on
    uint32_t rows[kTileM / 32];       // whose bit is clear take nothing of it, a NaN of the adapter's least of all
};

// One launch. Units are (row group, output tile) blocks of Y; a row group is one planner tile, or two
// that share the weight's tile on an SM pair (wide form).
struct Fp8Params {
    CUtensorMap inline_bmaps[kFp8InlineAdapters];   // B_a [d_out, rank] bf16 (inline work list)
    Tile inline_tiles[kInlineTiles];
    // mixed: on single CTAs a tile's u_row is its first expand, its adapter their number; on pairs some tiles are kApart
    Fp8Expand expand[kFp8Expands];
    int mixed;
    int inline_wl;
    CUtensorMap tm_x;                 // X [T, d_in] e4m3, box 128 x a_rows, 128-byte swizzle
    CUtensorMap tm_w;                 // W [d_out, d_in] e4m3, box 128 x tile_n, on pairs 128 x 64
    CUtensorMap tm_u;                 // U [u_rows, rank] bf16, box 64 x a_rows
    CUtensorMap tm_y;                 // Y [T, d_out] bf16, box 64 x 32, 128-byte swizzle; single CTAs 32 x 32, 64-byte
    const CUtensorMap* tm_b;          // device array per compact adapter (when not inline)
    const Tile* tiles;                // device array (when not inline)
    const float* xs;                  // [T, k_blocks]
    const float* ws;                  // [ceil(d_out / 128), k_blocks]
    void* y;                          // [T, d_out] bf16
    int* status;
    unsigned long long wait_limit_ns;
    int n_groups;                     // row groups
    int n_ntiles, tile_n;             // output tiles: 128 or 256 columns; 256 in the wide form
    int raster_group;                 // column tiles whose row groups run before the next column tiles
    int k_blocks;                     // ceil(d_in / 128)
    int k_lora;                       // ceil(rank / 64)
    int lora_stages;                  // of an expand's block: all k_lora where the ring is long enough, else a part of them
    int most_expands;                 // of a unit
    int expand_blocks;                // of an expand: k_lora / lora_stages
    int d_out;
    int parts;                        // K parts of a unit (1 in the wide form)
    int a_rows;                       // rows of an A box: 128, or fewer (a multiple of 16) for a batch of one tile
    int stages;
    int rows;                         // T
    int vec_scales;                   // both scales' rows are 16-byte aligned
    int chained;                      // may begin while the stream's kernel before it ends
    int late_u;                       // (chained) beside the call's own shrink, which it waits for ahead of U alone
    int wide;                         // SM pairs, 256 x 256 blocks, persistent
    int debug_stall;
};

// The adapters' shrink ahead of it, U[t, :] = bf16(s_a X[t, :] A_a^T), for batches of few tiles: a tile's K is split over
// the CTAs of a cluster, so that a few tiles find most SMs.
constexpr int kShrinkThreads = 256;   // warp 0 TMA, 1 MMA, 2 owns TMEM, 4..7 epilogue
struct ShrinkParams {
    CUtensorMap inline_amaps[kFp8InlineAdapters];   // A_a [rank, d_in] bf16, box 64 x n
    Tile inline_tiles[kInlineTiles];
    int32_t inline_seg[2 * kInlineSegs + 1];     // merged segments: offsets, then compact ids
    float inline_scales[kFp8InlineAdapters];
    int inline_wl;
    CUtensorMap tm_x;                 // X [T, d_in] bf16, box 64 x 128
    const CUtensorMap* tm_a;          // device arrays (when not inline)
    const Tile* tiles;
    const int32_t* seg_off;
    const int32_t* seg_id;
    const float* scales;
    void* u;                          // [u_rows, rank] bf16; a tile's rows from its u_row on
    int* status;
    unsigned long long wait_limit_ns;
    int n_tiles, n_seg, rank;
    int n, rank_tiles;                // columns of a unit, a multiple of 16; units side by side
    int k_steps;                      // ceil(d_in / 64)
    int parts, stages, chained, debug_stall;
};

// kernels_fp8.cu
// The most stages of as many blocks in a row as there are TMEM buffers, where units of nk base blocks (a stage each) and
// `expands` blocks of `lora_stages` follow one another: the ring is at least as long (the issuing warps' comment).
int fp8_window(int bufs, int nk, int expands, int lora_stages);
int shrink_stages(int n);
cudaError_t launch_shrink(const ShrinkParams& p, int grid, cudaStream_t stream);
size_t fp8_smem_bytes(int wide, int tile_n, int a_rows, int stages);
int fp8_max_clusters(int tile_n, int parts);
cudaError_t fp8_prepare_device();
cudaError_t launch_fp8(const Fp8Params& p, int grid, cudaStream_t stream);

}  // namespace lora
