/*
 * lora_layer.h -- the operators between the projections of an adapted layer, on one GB300
 * (sm_103a): the residual's addition with the root-mean-square norm ahead of a projection, the
 * append of new keys and values to a paged cache, and attention of the batch's new rows over
 * that cache, with an optional sliding window and first tokens that stay visible (sinks); the gated
 * activation, rows and weights in 8 bits, for 8-bit projections (lora_linear_forward_fp8); and, behind
 * the last projection, log probabilities of given tokens.
 *
 * They serve the same batches as lora_linear_forward: rows grouped into request segments, a few
 * chats with 1 to 8 new rows each beside prompts of thousands. `q_offsets` below is the host
 * array that lora_linear_forward takes as seg_offsets. What grows from step to step (cache
 * lengths, page tables) is read on the device, so that a decode step captured in a CUDA graph
 * can be replayed as the caches grow.
 *
 * Types: activations and caches are bf16; sums, softmax statistics and norms are held in fp32;
 * every output is rounded once (round to nearest even), except that the softmax weights are
 * rounded to bf16 for the tensor-core product with V (their sum is taken before that rounding).
 * Strides are in elements. Every pointer to bf16 or 8-bit data is 16-byte aligned and every
 * stride a multiple of 8 elements; the innermost axis is contiguous.
 *
 * Errors, streams and codes are those of lora_linear.h: arguments are checked on the host before
 * any launch, a failed check launches nothing and leaves outputs untouched, calls are enqueued
 * on `stream` and return without waiting (their kernels may be scheduled while the stream's kernel
 * before them ends, and wait for it before they touch memory or let the next one begin). Values that live on the device
 * (cache lengths, page tables) cannot be checked there: a length is used as if clamped to
 * [0, pages x page_size], and a page number outside [0, n_pages) is read as zeros and never written.
 */
#ifndef LORA_LAYER_H
#define LORA_LAYER_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_LAYER_MAX_WIDTH 32768 /* features of a normalised row */
#define LORA_LAYER_MAX_SEQS 1024   /* sequences of one call */
#define LORA_LAYER_MAX_TOP 32      /* alternatives of a row of logits */
#define LORA_LAYER_MAX_VOCAB (1 << 24) /* entries of a row of logits */
#define LORA_LAYER_MAX_CONTEXT (1 << 27) /* pages_per_seq x page_size: tokens a sequence's table can hold */

/*
 * lora_linear_add_rms_norm -- for every row t of x [rows, width]:
 *     h = x + residual                       (h = x where residual is NULL)
 *     y = h * (mean(h^2) + eps)^(-1/2) * (weight + weight_offset)
 * The norm is taken of the unrounded fp32 sum h.
 *   x, x_stride                device bf16 [rows, width]: row stride >= width.
 *   residual, residual_stride  device bf16 [rows, width], or NULL.
 *   weight                     device bf16 [width].
 *   h_out, h_stride            device bf16 [rows, width]: h rounded; NULL = not written. May be
 *                              `residual` or `x` itself (same pointer and stride).
 *   y, y_stride                device bf16 [rows, width], or NULL. May be `x` itself.
 *   q8, q8_stride              device e4m3 [rows, width], or NULL: y in 8 bits,
 *                              q = e4m3(y r) (nearest even, saturating) with r = 1 / s rounded to
 *                              fp32: beside a tie the code may be y / s's neighbour,
 *   scales, group              s = max(max|y| / 448, 2^-100), fp32: over the whole row
 *                              (group 0, scales [rows]) or over every `group` features
 *                              (32, 64, 128 or 256; scales [rows, ceil(width / group)], the last
 *                              group may be short). At least one of y and q8 is given.
 *   rows >= 0; width a multiple of 8 in [8, LORA_LAYER_MAX_WIDTH]; eps >= 0, finite.
 * No other overlap between an output and another buffer is allowed. A row with a NaN or an
 * infinity gives NaN in that row alone.
 */
int lora_linear_add_rms_norm(const void* x, long long x_stride, const void* residual, long long residual_stride,
                             const void* weight, float weight_offset, float eps, int rows, int width,
                             void* h_out, long long h_stride, void* y, long long y_stride,
                             void* q8, long long q8_stride, float* scales, int group, void* stream);

/*
 * lora_linear_silu_mul -- the gated activation between the gate_up and down projections, for every row t:
 *     y = g / (1 + e^(-g)) * u,   g = x[t, 0 : width], u = x[t, width : 2 width]
 *   x, x_stride    device bf16 [rows, 2 width]: row stride >= 2 width.
 *   y, y_stride    device bf16 [rows, width], or NULL.
 *   q8, q8_stride, scales, group   device e4m3 [rows, width], or NULL: y in 8 bits, as lora_linear_add_rms_norm's.
 *                  At least one of y and q8 is given; both are for a projection whose adapters read bf16.
 *   rows >= 0; width a multiple of 8 in [8, LORA_LAYER_MAX_WIDTH]. No output may overlap another buffer.
 * A NaN or an infinity gives a NaN or a scale of infinity in its row's group (group 0: its row) alone.
 */
int lora_linear_silu_mul(const void* x, long long x_stride, int rows, int width, void* y, long long y_stride,
                         void* q8, long long q8_stride, float* scales, int group, void* stream);

/*
 * lora_linear_fp8_rows -- rows of bf16 in 8 bits: q8, scales and group as lora_linear_add_rms_norm writes them for y = x.
 *   x, x_stride    device bf16 [rows, width]; limits as lora_linear_silu_mul.
 */
int lora_linear_fp8_rows(const void* x, long long x_stride, int rows, int width, void* q8, long long q8_stride,
                         float* scales, int group, void* stream);

/*
 * lora_linear_fp8_blocks -- a weight in 8 bits, for lora_linear_forward_fp8; run once when it is loaded.
 *   w, w_stride    device bf16 [rows, cols]: rows >= 0, cols a multiple of 8, both at most LORA_MAX_FEATURES.
 *   q8, q8_stride  device e4m3 [rows, cols]: q = e4m3(w r), r = 1 / s rounded to fp32 (nearest even, saturating).
 *   scales         device fp32 [ceil(rows / 128), ceil(cols / 128)], contiguous: s = max(max|w| / 448, 2^-100) over
 *                  every block of 128 x 128 (the last ones may be smaller); / 448 is a product with 1 / 448 in fp32.
 * No output may overlap another buffer. A NaN or an infinity leaves nothing of its block.
 */
int lora_linear_fp8_blocks(const void* w, long long w_stride, int rows, int cols, void* q8, long long q8_stride,
                           float* scales, void* stream);

/*
 * lora_linear_token_logprobs -- for every row of logits x, with z = x / temperature:
 *   logprobs[t]     z_i - log sum_j e^(z_j) of the given token i = tokens[t]; NaN where i is not in [0, vocab).
 *   ranks[t]        entries before i in the order of falling x, ties by rising index (0: the most likely); -1 there.
 *   entropy[t]      -sum_j p_j log p_j, p = softmax(z), in nats.
 *   top_logprobs, top_tokens   [rows, top]: the first `top` entries of that order.
 *   logits, stride  device bf16 (is_fp32 0) or fp32 (1) [rows, vocab], row stride >= vocab elements; no alignment
 *                   beyond the element's. Entries of -inf (tokens ruled out) have probability 0.
 *   tokens          device int32 (tokens64 0) or int64 (1) [rows]; NULL where logprobs and ranks are.
 *   temperature     in [2^-64, 2^64].
 *   top             0 to LORA_LAYER_MAX_TOP, at most vocab.
 * Any of logprobs, ranks and entropy may be NULL, but not all outputs. They are contiguous and overlap nothing.
 * Sums, and the exponentials in them, are fp32. A row of -inf alone has log
 * probabilities of -inf and entropy 0; one with a NaN or +inf has NaN for both, and its ranks and alternatives go by
 * the order, in which a NaN is behind -inf. The same call gives the same bits.
 */
int lora_linear_token_logprobs(const void* logits, long long stride, int is_fp32, int rows, int vocab,
                               const void* tokens, int tokens64, float temperature, int top, float* logprobs,
                               int32_t* ranks, float* entropy, float* top_logprobs, int32_t* top_tokens, void* stream);

/*
 * The paged cache and the batch, as the calls below take them.
 *   k_cache, v_cache   device bf16, n_pages pages of page_size tokens with n_kv_heads heads of
 *                      head_dim each; element (page, token, head, i) is at page * page_stride +
 *                      token * token_stride + head * head_stride + i. Any order of the axes and
 *                      any interleaving of K and V that strides describe will do. Positive strides.
 *   page_size          a multiple of 16.
 *   block_table        device int32 [n_seqs, pages_per_seq], row stride `table_stride`: token j of
 *                      sequence s is at token j % page_size of page block_table[s][j / page_size].
 *   kv_lens            device int32 [n_seqs]: tokens of each sequence, the new ones included.
 *   q_offsets          HOST int32 [n_seqs + 1]: q_offsets[0] = 0, nondecreasing; the new rows of
 *                      sequence s are [q_offsets[s], q_offsets[s + 1]) and are its last tokens:
 *                      row i has position kv_lens[s] - q_len + i. A row whose position is
 *                      negative sees nothing and is not appended.
 */
typedef struct lora_kv_cache {
    void* k;
    void* v;
    long long k_page_stride, k_token_stride, k_head_stride;
    long long v_page_stride, v_token_stride, v_head_stride;
    int n_pages, page_size, n_kv_heads, head_dim;
    const int32_t* block_table;
    long long table_stride;
    int pages_per_seq, n_seqs;
    const int32_t* kv_lens;
    const int32_t* q_offsets;
} lora_kv_cache;

/*
 * lora_linear_kv_append -- writes the new rows' keys and values to their places in the cache,
 * turning queries and keys by their position first (rotary embedding, halves layout):
 *     (a_i, b_i) -> (a_i cos - b_i sin, b_i cos + a_i sin),  a = x[0 : rot/2], b = x[rot/2 : rot]
 * with cos, sin at [position][i]; features rot and up are copied.
 *   q, q_stride, q_head_stride          device bf16 [T, n_heads, head_dim], or NULL with q_out.
 *   q_out, qo_stride, qo_head_stride    device bf16; may be q itself (same strides), and shares no place with k
 *                                       or v (which may lie beside it, as slices of one buffer).
 *   k, v and their strides              device bf16 [T, n_kv_heads, head_dim].
 *   cos, sin           device fp32 [n_positions, rot / 2], contiguous, 16-byte aligned; NULL when rot = 0. A
 *                      position past the last row uses the last one, a negative one (a query before its
 *                      sequence's start, which is turned all the same) the first.
 *   rot                0, or a multiple of 16 up to head_dim.
 *   head_dim           a multiple of 8 up to 512; n_heads >= 0.
 * T = q_offsets[n_seqs]. Two rows never write one place unless a page is listed twice.
 */
int lora_linear_kv_append(const lora_kv_cache* cache, const void* q, long long q_stride, long long q_head_stride,
                          void* q_out, long long qo_stride, long long qo_head_stride, int n_heads,
                          const void* k, long long k_stride, long long k_head_stride,
                          const void* v, long long v_stride, long long v_head_stride,
                          const float* cos, const float* sin, int rot, int n_positions, void* stream);

typedef struct lora_attn lora_attn; /* opaque handle: workspace of attention calls */

/*
 * lora_linear_attn_create -- a handle for attention with this head layout on one device.
 *   n_heads, n_kv_heads  n_heads a multiple of n_kv_heads, at most 128 query heads to a
 *                        key/value head.
 *   head_dim             64, 128 or 256.
 *   page_size            a multiple of 16 in [16, 2^20].
 *   max_tokens           most new rows of a call, in [1, LORA_MAX_TOKENS].
 *   max_seqs             most sequences of a call, in [1, LORA_LAYER_MAX_SEQS].
 * The handle owns its workspace (partial sums of split caches, a status word). Calls on one
 * handle must be ordered on one stream. Returns LORA_OK, LORA_EINVAL, LORA_ENODEV, LORA_ENOMEM
 * or LORA_ECUDA.
 */
int lora_linear_attn_create(lora_attn** out, int n_heads, int n_kv_heads, int head_dim, int page_size,
                            int max_tokens, int max_seqs, int device);

/*
 * lora_linear_attn_forward -- o[t] = sum_j p_tj v_j, p_t = softmax over the visible j of
 * scale * q_t . k_j, per query head; head n reads key/value head n / (n_heads / n_kv_heads).
 * A row at position p sees token j <= p if window = 0, or j > p - window, or j < sinks.
 * A row that sees no token gives zeros.
 *   q, out     device bf16 [T, n_heads, head_dim] with row and head strides; out must not
 *              overlap q or the cache.
 *   scale      > 0, finite.
 *   window     0 (none) or >= 1; sinks >= 0 (ignored when window = 0).
 * The cache holds the new rows' keys and values already (lora_linear_kv_append). What tokens hold
 * that no row of their sequence sees (at or past kv_lens, between the sinks and the window) is
 * never used; a NaN or infinity in the value of a token that one row of a sequence sees may also
 * reach rows of that sequence that do not see it.
 * Sequences of at most 16 rows per key/value head (q_len * n_heads / n_kv_heads) and longer ones
 * run in different kernels of the same call; the sums' order depends on the batch, so results of
 * one row in two batches may differ in the last bit. The same call gives the same bits.
 * May be recorded by stream capture.
 */
int lora_linear_attn_forward(lora_attn* h, const lora_kv_cache* cache, const void* q, long long q_stride,
                             long long q_head_stride, void* out, long long out_stride, long long out_head_stride,
                             float scale, int window, int sinks, void* stream);

/* lora_linear_attn_validate -- the host checks of lora_linear_attn_forward, without a handle or a GPU. */
int lora_linear_attn_validate(int n_heads, int n_kv_heads, int head_dim, int page_size, int max_tokens,
                              int max_seqs, const lora_kv_cache* cache, const void* q, long long q_stride,
                              long long q_head_stride, const void* out, long long out_stride,
                              long long out_head_stride, float scale, int window, int sinks);

/*
 * lora_linear_attn_set_option -- options of an attention handle, for later calls (anything else: LORA_EINVAL):
 *   LORA_OPT_WAIT_LIMIT_US   bound of every wait in a kernel, 1,000 to 60,000,000 microseconds (default 4,000,000).
 *   LORA_OPT_DEBUG_STALL     tests only: n > 0 = a block's load warp stops after n - 1 tiles of K and V, so that the
 *                            other warps' waits run out; 0 = off.
 */
int lora_linear_attn_set_option(lora_attn* h, int option, long long value);

/* lora_linear_attn_status -- LORA_OK, or LORA_ETIMEOUT if a kernel of this handle gave up a bounded wait (its
 * output is incomplete). Waits for the device first. reset != 0 clears the status word afterwards. */
int lora_linear_attn_status(lora_attn* h, int reset);

/* lora_linear_attn_destroy -- wait for the handle's device, free everything it owns. NULL-safe. */
int lora_linear_attn_destroy(lora_attn* h);

#ifdef __cplusplus
}
#endif

#endif /* LORA_LAYER_H */
