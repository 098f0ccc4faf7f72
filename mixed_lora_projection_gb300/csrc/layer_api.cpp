// C-ABI of the operators between the projections (include/lora_layer.h): argument checks, the
// attention handle and its workspace, launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "../../include/lora_layer.h"
#include "layer_internal.h"

using namespace lora;

static_assert(kMaxSeqs == LORA_LAYER_MAX_SEQS, "the kernels' sequence limit is the header's");

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The bytes that a strided buffer covers: `outer` rows of `extent` bytes, `stride` bytes apart; a row is `inner`
// vectors of `width` bytes, `step` bytes apart (0: one). A single row's vectors are the rows.
struct Span {
    uintptr_t first = 0, last = 0, stride = 0, extent = 0, step = 0, width = 0;
};
Span span(const void* p, long long outer, long long so, long long inner, long long si, long long width, int elem) {
    Span s;
    if (!p || outer <= 0 || inner <= 0) return s;
    if (outer == 1) {
        outer = inner;
        so = si;
        inner = 1;
    }
    s.first = reinterpret_cast<uintptr_t>(p);
    s.stride = outer > 1 ? (uintptr_t)(so * elem) : 0;
    s.step = inner > 1 ? (uintptr_t)(si * elem) : 0;
    s.width = (uintptr_t)(width * elem);
    s.extent = (uintptr_t)(((inner - 1) * si + width) * elem);
    s.last = s.first + (uintptr_t)(outer - 1) * s.stride + s.extent;
    return s;
}
// Whether two buffers may share a byte. Column slices of one row-strided buffer do not, nor vectors that lie beside
// one another within a row.
bool meet(const Span& a, const Span& b) {
    if (!(a.first < b.last && b.first < a.last)) return false;
    if (a.stride == 0 || a.stride != b.stride) return true;
    const uintptr_t d = a.first <= b.first ? (b.first - a.first) % a.stride : (a.stride - (a.first - b.first) % a.stride) % a.stride;
    if (d >= a.extent && d + b.extent <= a.stride) return false;
    if (a.step == 0 || a.step != b.step || a.stride % a.step) return true;
    const uintptr_t e = d % a.step;
    return !(e >= a.width && e + b.width <= a.step);
}

constexpr long long kMaxStride = 1ll << 38;   // elements: a tensor map's strides stay under 2^40 bytes

// A stride of `align` elements' multiple, large enough for rows of `least` elements.
bool stride_ok(long long s, long long least, int align) { return s >= least && s <= kMaxStride && s % align == 0; }

int check_offsets(const int32_t* off, int n, int* rows) {
    if (!off || off[0] != 0) return LORA_EINVAL;
    for (int i = 0; i < n; ++i)
        if (off[i + 1] < off[i]) return LORA_EINVAL;
    if (off[n] > LORA_MAX_TOKENS) return LORA_EINVAL;
    *rows = off[n];
    return LORA_OK;
}

int check_cache(const lora_kv_cache* c, int* rows) {
    if (!c || c->n_seqs < 1 || c->n_seqs > LORA_LAYER_MAX_SEQS) return LORA_EINVAL;
    if (check_offsets(c->q_offsets, c->n_seqs, rows) != LORA_OK) return LORA_EINVAL;
    if (c->n_kv_heads < 1 || c->n_kv_heads > 4096 || c->head_dim < 8 || c->head_dim > 512 || c->head_dim % 8) return LORA_EINVAL;
    if (c->page_size < 16 || c->page_size > (1 << 20) || c->page_size % 16) return LORA_EINVAL;
    if (c->n_pages < 1 || c->pages_per_seq < 1 || (long long)c->pages_per_seq * c->page_size > LORA_LAYER_MAX_CONTEXT) return LORA_EINVAL;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return LORA_EINVAL;
    const long long s[6] = {c->k_page_stride, c->k_token_stride, c->k_head_stride,
                            c->v_page_stride, c->v_token_stride, c->v_head_stride};
    for (long long v : s)
        if (!stride_ok(v, 8, 8)) return LORA_EINVAL;
    if (!c->block_table || !c->kv_lens || !aligned4(c->block_table) || !aligned4(c->kv_lens)) return LORA_EINVAL;
    if (c->table_stride < c->pages_per_seq || c->table_stride > (1ll << 31)) return LORA_EINVAL;
    return LORA_OK;
}

CacheView view(const lora_kv_cache* c) {
    CacheView v;
    v.k = c->k;
    v.v = c->v;
    v.k_page = c->k_page_stride;
    v.k_token = c->k_token_stride;
    v.k_head = c->k_head_stride;
    v.v_page = c->v_page_stride;
    v.v_token = c->v_token_stride;
    v.v_head = c->v_head_stride;
    v.table = c->block_table;
    v.kv_lens = c->kv_lens;
    v.table_stride = c->table_stride;
    v.n_pages = c->n_pages;
    v.page_size = c->page_size;
    v.n_kv = c->n_kv_heads;
    v.dim = c->head_dim;
    v.pages_per_seq = c->pages_per_seq;
    v.n_seqs = c->n_seqs;
    return v;
}

Span cache_span(const lora_kv_cache* c, bool v) {
    // pages, tokens and heads in any order: the far corner of the last element
    Span s;
    s.first = reinterpret_cast<uintptr_t>(v ? c->v : c->k);
    const long long far = (c->n_pages - 1) * (v ? c->v_page_stride : c->k_page_stride) +
                          (c->page_size - 1) * (v ? c->v_token_stride : c->k_token_stride) +
                          (c->n_kv_heads - 1) * (v ? c->v_head_stride : c->k_head_stride) + c->head_dim;
    s.last = s.first + (uintptr_t)far * 2;
    return s;
}

// The device's GPU is an sm_103 one (the kernels are compiled for nothing else).
int check_device(int device) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess) {
        cudaGetLastError();
        return LORA_ENODEV;
    }
    return major == 10 && minor == 3 ? LORA_OK : LORA_ENODEV;
}

int check_layout(int n_heads, int n_kv, int dim, int page_size, int max_tokens, int max_seqs) {
    if (n_kv < 1 || n_heads < n_kv || n_heads > 65536 || n_heads % n_kv || n_heads / n_kv > 128) return LORA_EINVAL;
    if (dim != 64 && dim != 128 && dim != 256) return LORA_EINVAL;
    if (page_size < 16 || page_size > (1 << 20) || page_size % 16) return LORA_EINVAL;
    if (max_tokens < 1 || max_tokens > LORA_MAX_TOKENS || max_seqs < 1 || max_seqs > LORA_LAYER_MAX_SEQS) return LORA_EINVAL;
    return LORA_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor map of a cache: 64 features of one head by `granule` tokens of one page, rows 128-byte
// swizzled. The axes past the features go by ascending stride, whatever the caller's layout;
// *order says which of (0 head, 1 token, 2 page) each of them is, two bits per axis.
bool encode_cache(EncodeTiledFn encode, CUtensorMap* m, int* order, const CacheView& c, bool v, int granule) {
    struct Axis {
        int what;
        uint64_t stride, size;
        uint32_t box;
    } ax[3] = {{0, (uint64_t)(v ? c.v_head : c.k_head), (uint64_t)c.n_kv, 1},
               {1, (uint64_t)(v ? c.v_token : c.k_token), (uint64_t)c.page_size, (uint32_t)granule},
               {2, (uint64_t)(v ? c.v_page : c.k_page), (uint64_t)c.n_pages, 1}};
    std::sort(ax, ax + 3, [](const Axis& a, const Axis& b) { return a.stride != b.stride ? a.stride < b.stride : a.what < b.what; });
    cuuint64_t dims[4] = {(cuuint64_t)c.dim, ax[0].size, ax[1].size, ax[2].size};
    cuuint64_t strides[3] = {ax[0].stride * 2, ax[1].stride * 2, ax[2].stride * 2};
    cuuint32_t box[4] = {64, ax[0].box, ax[1].box, ax[2].box};
    cuuint32_t step[4] = {1, 1, 1, 1};
    *order = ax[0].what | ax[1].what << 2 | ax[2].what << 4;
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v ? c.v : c.k, dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  // a head of 64 is 128 bytes of a token: wider fetches would bring in its neighbour
                  c.dim == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of the queries: 64 features of `group` heads by `tokens` rows, 128-byte swizzled; the axes past
// the features by ascending stride.
bool encode_queries(EncodeTiledFn encode, CUtensorMap* m, bool outer, const AttnParams& a, int dim, int group, int tokens) {
    const cuuint64_t heads = (cuuint64_t)a.n_heads, rows = (cuuint64_t)a.rows;
    cuuint64_t dims[3] = {(cuuint64_t)dim, outer ? rows : heads, outer ? heads : rows};
    const cuuint64_t sh = (cuuint64_t)a.q_head * 2, sr = (cuuint64_t)a.q_stride * 2;
    cuuint64_t strides[2] = {outer ? sr : sh, outer ? sh : sr};
    cuuint32_t box[3] = {64, (cuuint32_t)(outer ? tokens : group), (cuuint32_t)(outer ? group : tokens)};
    cuuint32_t step[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Makes `device` current for the life of a call.
struct DeviceGuard {
    int prev = -1;
    bool changed = false, ok = true;
    explicit DeviceGuard(int device) {
        ok = cudaGetDevice(&prev) == cudaSuccess;
        if (ok && prev != device) ok = changed = cudaSetDevice(device) == cudaSuccess;
    }
    ~DeviceGuard() {
        if (changed) cudaSetDevice(prev);
    }
};

}  // namespace

struct lora_attn {
    int device = 0, n_heads = 0, n_kv = 0, dim = 0, page_size = 0, max_tokens = 0, max_seqs = 0;
    int num_sms = 0;
    int* status = nullptr;              // status word; then the prompt kernel's two counters
    unsigned long long wait_limit_ns = 4000000000ull;
    int debug_stall = 0;
    EncodeTiledFn encode = nullptr;
    float* part_o = nullptr;            // sums of split units, their maxima and sums of weights
    float2* part_ml = nullptr;
    uint32_t* prefix = nullptr;         // sums of tiles: the decode kernel's, then the prompt kernel's
};

namespace {

// Everything a handle needs beside itself, on its device (which is current).
int set_up(lora_attn* h) {
    if (cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) return LORA_ENODEV;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
        return LORA_ECUDA;
    h->encode = reinterpret_cast<EncodeTiledFn>(fn);
    if (decode_prepare_device() != cudaSuccess || prompt_prepare_device() != cudaSuccess) return LORA_ECUDA;
    // two parts a block: of 16 rows (two decode blocks share an SM), or of a prompt unit's rows
    const size_t parts = 2 * (size_t)h->num_sms * std::max(2 * kDecodeRows, kPromptTile * prompt_tiles(h->dim));
    if (cudaMalloc(reinterpret_cast<void**>(&h->status), 3 * sizeof(int)) != cudaSuccess ||
        cudaMalloc(reinterpret_cast<void**>(&h->part_o), parts * h->dim * sizeof(float)) != cudaSuccess ||
        cudaMalloc(reinterpret_cast<void**>(&h->part_ml), parts * sizeof(float2)) != cudaSuccess ||
        cudaMalloc(reinterpret_cast<void**>(&h->prefix), (h->max_seqs + 1 + kPromptBlocks + 2) * sizeof(uint32_t)) != cudaSuccess)
        return LORA_ENOMEM;
    return cudaMemset(h->status, 0, 3 * sizeof(int)) == cudaSuccess ? LORA_OK : LORA_ECUDA;
}

// The decode kernel on the sequences of `list` (at most kDecodeRows rows per key/value head each).
int run_decode(lora_attn* h, const AttnParams& a, const SeqList<kMaxSeqs>& list) {
    DecodeParams p;
    p.a = a;
    p.group = h->n_heads / h->n_kv;
    p.granule = 64;                              // a power of two that divides the tile and the page
    while (h->page_size % p.granule) p.granule /= 2;
    p.slots = 16;
    while (p.slots > 2 && decode_smem(h->dim, p.slots, list.n) > kSmemTwo) --p.slots;
    p.grid = 2 * h->num_sms;
    p.most_rows = 0;
    for (int i = 0; i < list.n; ++i) p.most_rows = std::max(p.most_rows, (int)list.q_len[i] * p.group);
    p.part_o = h->part_o;
    p.part_ml = h->part_ml;
    p.prefix = h->prefix;
    if (!encode_cache(h->encode, &p.tm_k, &p.k_order, a.c, false, p.granule) ||
        !encode_cache(h->encode, &p.tm_v, &p.v_order, a.c, true, p.granule))
        return LORA_EINVAL;
    return launch_decode(p, list, a.stream) == cudaSuccess ? LORA_OK : LORA_ECUDA;
}

// The prompt kernel on the sequences of `list`.
int run_prompts(lora_attn* h, const AttnParams& a, PromptList<kMaxSeqs>& list) {
    PromptParams p;
    p.a = a;
    p.group = h->n_heads / h->n_kv;
    p.tile_tokens = kPromptTile / p.group;
    p.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.o_stride % 16 == 0 && a.o_head % 16 == 0;
    p.granule = 64;
    while (h->page_size % p.granule) p.granule /= 2;
    p.q_outer = a.q_head > a.q_stride;
    int most = 0;
    for (int i = 0; i < list.n; ++i) most = std::max(most, (int)list.q_len[i]);
    p.tiles = most > p.tile_tokens ? prompt_tiles(h->dim) : 1;
    const int step = p.tiles * p.tile_tokens;
    long long units = 0;
    for (int i = 0; i < list.n; ++i) {
        list.unit0[i] = (int32_t)units;
        units += (long long)((list.q_len[i] + step - 1) / step) * h->n_kv;
        if (units > 0x7fffffff / 8) return LORA_EUNSUPPORTED;
    }
    p.units = (int)units;
    p.blocks = std::min(h->num_sms, kPromptBlocks);
    // rows that a unit may have: those of the longest sequence where they fit the first tile, else all
    p.join_rows = most > p.tile_tokens ? p.tiles * kPromptTile : p.q_outer ? p.tile_tokens * p.group : most * p.group;
    p.whole = (int)(units / p.blocks * p.blocks);
    p.prefix = h->prefix + h->max_seqs + 1;
    p.counter = h->status + 1;
    p.part_o = h->part_o;
    p.part_ml = h->part_ml;
    if (!encode_cache(h->encode, &p.tm_k, &p.k_order, a.c, false, p.granule) ||
        !encode_cache(h->encode, &p.tm_v, &p.v_order, a.c, true, p.granule) ||
        !encode_queries(h->encode, &p.tm_q, p.q_outer, a, h->dim, p.group, p.tile_tokens))
        return LORA_EINVAL;
    return launch_prompt(p, list, a.stream) == cudaSuccess ? LORA_OK : LORA_ECUDA;
}

}  // namespace

extern "C" int lora_linear_add_rms_norm(const void* x, long long x_stride, const void* residual,
                                        long long residual_stride, const void* weight, float weight_offset, float eps,
                                        int rows, int width, void* h_out, long long h_stride, void* y,
                                        long long y_stride, void* q8, long long q8_stride, float* scales, int group,
                                        void* stream) {
    if (rows < 0 || width < 8 || width > LORA_LAYER_MAX_WIDTH || width % 8) return LORA_EINVAL;
    if (!isfinite(eps) || eps < 0.f || !isfinite(weight_offset)) return LORA_EINVAL;
    if (rows == 0) return LORA_OK;
    if (!x || !weight || (!y && !q8)) return LORA_EINVAL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h_out) || !aligned16(y) || !aligned16(q8))
        return LORA_EINVAL;
    if (!stride_ok(x_stride, width, 8) || (residual && !stride_ok(residual_stride, width, 8)) ||
        (h_out && !stride_ok(h_stride, width, 8)) || (y && !stride_ok(y_stride, width, 8)))
        return LORA_EINVAL;
    if (q8) {
        if (width % 8 || !stride_ok(q8_stride, width, 8) || !scales || !aligned4(scales)) return LORA_EINVAL;
        if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256) return LORA_EINVAL;
    }
    const Span sx = span(x, rows, x_stride, 1, 0, width, 2), sr = span(residual, rows, residual_stride, 1, 0, width, 2);
    const Span sw = span(weight, 1, 0, 1, 0, width, 2);
    const Span sh = span(h_out, rows, h_stride, 1, 0, width, 2), sy = span(y, rows, y_stride, 1, 0, width, 2);
    const Span sq = span(q8, rows, q8_stride, 1, 0, width, 1);
    const Span ss = q8 ? span(scales, rows, group ? (width + group - 1) / group : 1, 1, 0, group ? (width + group - 1) / group : 1, 4)
                       : Span();
    const Span outs[4] = {sh, sy, sq, ss};
    for (int i = 0; i < 4; ++i) {
        if (meet(outs[i], sw)) return LORA_EINVAL;
        for (int k = i + 1; k < 4; ++k)
            if (meet(outs[i], outs[k])) return LORA_EINVAL;
        // a row is read whole before its outputs are written, so h or y may be an input itself
        const bool is_x = (i == 0 && h_out == x && h_stride == x_stride) || (i == 1 && y == x && y_stride == x_stride);
        const bool is_r = residual && i == 0 && h_out == residual && h_stride == residual_stride;
        if ((!is_x && meet(outs[i], sx)) || (!is_r && meet(outs[i], sr))) return LORA_EINVAL;
    }
    NormParams p;
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.h = h_out;
    p.y = y;
    p.q8 = q8;
    p.scales = scales;
    p.x_stride = x_stride;
    p.r_stride = residual_stride;
    p.h_stride = h_stride;
    p.y_stride = y_stride;
    p.q8_stride = q8_stride;
    p.weight_offset = weight_offset;
    p.eps = eps;
    p.rows = rows;
    p.width = width;
    p.group = group;
    return launch_add_rms_norm(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK : LORA_ECUDA;
}

extern "C" int lora_linear_kv_append(const lora_kv_cache* cache, const void* q, long long q_stride,
                                     long long q_head_stride, void* q_out, long long qo_stride,
                                     long long qo_head_stride, int n_heads, const void* k, long long k_stride,
                                     long long k_head_stride, const void* v, long long v_stride,
                                     long long v_head_stride, const float* cos, const float* sin, int rot,
                                     int n_positions, void* stream) {
    int rows = 0;
    if (check_cache(cache, &rows) != LORA_OK) return LORA_EINVAL;
    const int dim = cache->head_dim, n_kv = cache->n_kv_heads;
    if (n_heads < 0 || n_heads > 65536 || rot < 0 || rot > dim || rot % 16) return LORA_EINVAL;
    if (rot && (!cos || !sin || n_positions < 1 || !aligned16(cos) || !aligned16(sin))) return LORA_EINVAL;
    if (rows == 0) return LORA_OK;
    if ((q == nullptr) != (q_out == nullptr) || (q && n_heads < 1)) return LORA_EINVAL;
    if (!k || !v || !aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v)) return LORA_EINVAL;
    if (q && (!stride_ok(q_stride, dim, 8) || !stride_ok(q_head_stride, dim, 8) || !stride_ok(qo_stride, dim, 8) ||
              !stride_ok(qo_head_stride, dim, 8)))
        return LORA_EINVAL;
    if (!stride_ok(k_stride, dim, 8) || !stride_ok(k_head_stride, dim, 8) || !stride_ok(v_stride, dim, 8) ||
        !stride_ok(v_head_stride, dim, 8))
        return LORA_EINVAL;
    const Span kc = cache_span(cache, false), vc = cache_span(cache, true);
    const Span sq = span(q, rows, q_stride, n_heads, q_head_stride, dim, 2);
    const Span so = span(q_out, rows, qo_stride, n_heads, qo_head_stride, dim, 2);
    const Span sk = span(k, rows, k_stride, n_kv, k_head_stride, dim, 2);
    const Span sv = span(v, rows, v_stride, n_kv, v_head_stride, dim, 2);
    if (meet(kc, sq) || meet(kc, sk) || meet(kc, sv) || meet(vc, sq) || meet(vc, sk) || meet(vc, sv) || meet(kc, so) ||
        meet(vc, so))
        return LORA_EINVAL;
    const bool in_place = q && q == q_out && q_stride == qo_stride && q_head_stride == qo_head_stride;
    // (q, k and v may be slices of one buffer)
    if (q && ((!in_place && meet(so, sq)) || meet(so, sk) || meet(so, sv))) return LORA_EINVAL;
    AppendParams p;
    p.c = view(cache);
    p.q = q;
    p.q_out = q_out;
    p.k = k;
    p.v = v;
    p.cos = cos;
    p.sin = sin;
    p.q_stride = q_stride;
    p.q_head = q_head_stride;
    p.qo_stride = qo_stride;
    p.qo_head = qo_head_stride;
    p.k_stride = k_stride;
    p.k_head = k_head_stride;
    p.v_stride = v_stride;
    p.v_head = v_head_stride;
    p.n_heads = n_heads;
    p.rot = rot;
    p.n_positions = n_positions;
    p.rows = rows;
    return launch_kv_append(p, cache->q_offsets, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK : LORA_ECUDA;
}

extern "C" int lora_linear_attn_validate(int n_heads, int n_kv_heads, int head_dim, int page_size, int max_tokens,
                                         int max_seqs, const lora_kv_cache* cache, const void* q, long long q_stride,
                                         long long q_head_stride, const void* out, long long out_stride,
                                         long long out_head_stride, float scale, int window, int sinks) {
    int rows = 0;
    if (check_layout(n_heads, n_kv_heads, head_dim, page_size, max_tokens, max_seqs) != LORA_OK) return LORA_EINVAL;
    if (check_cache(cache, &rows) != LORA_OK) return LORA_EINVAL;
    if (cache->n_kv_heads != n_kv_heads || cache->head_dim != head_dim || cache->page_size != page_size) return LORA_EINVAL;
    if (cache->n_seqs > max_seqs || rows > max_tokens) return LORA_EINVAL;
    if (!isfinite(scale) || !(scale > 0.f) || window < 0 || sinks < 0) return LORA_EINVAL;
    if (rows == 0) return LORA_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out)) return LORA_EINVAL;
    if (!stride_ok(q_stride, head_dim, 8) || !stride_ok(q_head_stride, head_dim, 8) || !stride_ok(out_stride, head_dim, 8) ||
        !stride_ok(out_head_stride, head_dim, 8))
        return LORA_EINVAL;
    const Span so = span(out, rows, out_stride, n_heads, out_head_stride, head_dim, 2);
    if (meet(so, span(q, rows, q_stride, n_heads, q_head_stride, head_dim, 2)) || meet(so, cache_span(cache, false)) ||
        meet(so, cache_span(cache, true)))
        return LORA_EINVAL;
    return LORA_OK;
}

extern "C" int lora_linear_attn_create(lora_attn** out, int n_heads, int n_kv_heads, int head_dim, int page_size,
                                       int max_tokens, int max_seqs, int device) {
    if (!out) return LORA_EINVAL;
    *out = nullptr;
    if (check_layout(n_heads, n_kv_heads, head_dim, page_size, max_tokens, max_seqs) != LORA_OK) return LORA_EINVAL;
    int rc = check_device(device);
    if (rc != LORA_OK) return rc;
    lora_attn* h = new (std::nothrow) lora_attn;
    if (!h) return LORA_ENOMEM;
    h->device = device;
    h->n_heads = n_heads;
    h->n_kv = n_kv_heads;
    h->dim = head_dim;
    h->page_size = page_size;
    h->max_tokens = max_tokens;
    h->max_seqs = max_seqs;
    DeviceGuard guard(device);
    rc = guard.ok ? set_up(h) : LORA_ENODEV;
    if (rc != LORA_OK) {
        cudaGetLastError();
        lora_linear_attn_destroy(h);
        return rc;
    }
    *out = h;
    return LORA_OK;
}

extern "C" int lora_linear_attn_forward(lora_attn* h, const lora_kv_cache* cache, const void* q, long long q_stride,
                                        long long q_head_stride, void* out, long long out_stride,
                                        long long out_head_stride, float scale, int window, int sinks, void* stream) {
    if (!h) return LORA_EINVAL;
    if (lora_linear_attn_validate(h->n_heads, h->n_kv, h->dim, h->page_size, h->max_tokens, h->max_seqs, cache, q, q_stride,
                                  q_head_stride, out, out_stride, out_head_stride, scale, window, sinks) != LORA_OK)
        return LORA_EINVAL;
    const int rows = cache->q_offsets[cache->n_seqs];
    if (rows == 0) return LORA_OK;
    DeviceGuard guard(h->device);
    if (!guard.ok) return LORA_ECUDA;
    AttnParams p;
    p.c = view(cache);
    p.q = q;
    p.out = out;
    p.q_stride = q_stride;
    p.q_head = q_head_stride;
    p.o_stride = out_stride;
    p.o_head = out_head_stride;
    p.n_heads = h->n_heads;
    p.rows = rows;
    p.window = std::min(window, 2 * LORA_LAYER_MAX_CONTEXT);       // longer than any sequence: the same, and no overflow
    p.sinks = window ? std::min(sinks, LORA_LAYER_MAX_CONTEXT) : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = h->status;
    p.wait_limit_ns = h->wait_limit_ns;
    p.debug_stall = h->debug_stall;
    p.stream = static_cast<cudaStream_t>(stream);
    // sequences with few rows and long ones go to different kernels
    const int g = h->n_heads / h->n_kv;
    SeqList<kMaxSeqs> few;
    SeqList<kMaxSeqs> many;
    few.n = many.n = 0;
    for (int i = 0; i < cache->n_seqs; ++i) {
        const int n = cache->q_offsets[i + 1] - cache->q_offsets[i];
        if (n == 0) continue;
        SeqList<kMaxSeqs>& l = (long long)n * g > kDecodeRows ? many : few;
        l.seq[l.n] = (uint16_t)i;
        l.row[l.n] = cache->q_offsets[i];
        l.q_len[l.n++] = n;
    }
    if (many.n) {
        // the sequences with most rows first: the last blocks of a launch had better be short
        int by[kMaxSeqs];
        for (int i = 0; i < many.n; ++i) by[i] = i;
        std::sort(by, by + many.n, [&](int a, int b) { return many.q_len[a] != many.q_len[b] ? many.q_len[a] > many.q_len[b] : a < b; });
        PromptList<kMaxSeqs> sorted;
        sorted.n = many.n;
        for (int i = 0; i < many.n; ++i) {
            sorted.seq[i] = many.seq[by[i]];
            sorted.row[i] = many.row[by[i]];
            sorted.q_len[i] = many.q_len[by[i]];
        }
        const int rc = run_prompts(h, p, sorted);
        if (rc != LORA_OK) return rc;
    }
    return few.n ? run_decode(h, p, few) : LORA_OK;
}

extern "C" int lora_linear_attn_set_option(lora_attn* h, int option, long long value) {
    if (!h) return LORA_EINVAL;
    switch (option) {
        case LORA_OPT_WAIT_LIMIT_US:
            if (value < 1000 || value > 60000000) return LORA_EINVAL;
            h->wait_limit_ns = (unsigned long long)value * 1000ull;
            return LORA_OK;
        case LORA_OPT_DEBUG_STALL:
            if (value < 0 || value > kNoStall) return LORA_EINVAL;
            h->debug_stall = (int)value;
            return LORA_OK;
        default:
            return LORA_EINVAL;
    }
}

extern "C" int lora_linear_attn_status(lora_attn* h, int reset) {
    if (!h) return LORA_EINVAL;
    int v = 0;
    DeviceGuard guard(h->device);
    if (!guard.ok) return LORA_ECUDA;
    int rc = LORA_OK;
    if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(&v, h->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        rc = LORA_ECUDA;
    else if (reset && cudaMemset(h->status, 0, sizeof(int)) != cudaSuccess)
        rc = LORA_ECUDA;
    return rc != LORA_OK ? rc : v ? LORA_ETIMEOUT : LORA_OK;
}

extern "C" int lora_linear_attn_destroy(lora_attn* h) {
    if (!h) return LORA_OK;
    {
        DeviceGuard guard(h->device);
        if (guard.ok) {
            cudaDeviceSynchronize();
            cudaFree(h->status);
            cudaFree(h->part_o);
            cudaFree(h->part_ml);
            cudaFree(h->prefix);
        }
    }
    delete h;
    return LORA_OK;
}
