// kvq_internal.h -- launchers shared between the kernel files and the C ABI layer.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq.h"

namespace kvq {

// Byte offsets of the four sections of a (page, kv-head) block.
struct BlockLayout {
    int32_t d, P, Gk, Gv;
    int32_t v_codes;   // P * d / 2
    int32_t k_scales;  // P * d
    int32_t v_scales;  // P * d + P * (d / Gk) * 2
    int32_t bytes;     // padded to 16
};

inline BlockLayout block_layout(const kvq_cache_config& c) {
    BlockLayout L;
    L.d = c.head_dim;
    L.P = c.page_size;
    L.Gk = c.group_k;
    L.Gv = c.group_v;
    L.v_codes = c.page_size * c.head_dim / 2;
    L.k_scales = c.page_size * c.head_dim;
    L.v_scales = L.k_scales + c.page_size * (c.head_dim / c.group_k) * 2;
    const int32_t raw = L.v_scales + c.page_size * (c.head_dim / c.group_v) * 2;
    L.bytes = (raw + 15) / 16 * 16;
    return L;
}

// Division of 32-bit n < 2^31 by a fixed divisor d >= 1 as a multiply-high, add and
// shift: with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (umulhi(n, m) + n) >> l, and the sum stays below 2^32 because n < 2^31.
struct FastDiv {
    uint32_t d, m, l;
};
inline FastDiv make_fastdiv(uint32_t d) {
    FastDiv f;
    f.d = d;
    f.l = 0;
    while ((1ull << f.l) < d) ++f.l;
    f.m = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.l) - d)) / d + 1);
    return f;
}
#ifdef __CUDACC__
__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
    return (__umulhi(n, f.m) + n) >> f.l;
}
#endif

struct QuantizeArgs {
    uint8_t* pool;
    const __half* k;
    const __half* v;
    const int32_t* block_table;
    const int32_t* start_pos;
    // ragged batches: sequence b owns tokens cu_rows[b] .. cu_rows[b + 1] - 1 of the row
    // arrays (nullptr: every sequence owns n_new tokens, sequence b from b * n_new)
    const int32_t* cu_rows;
    uint32_t* status;
    int32_t max_blocks, B, n_new, Hkv, num_pages;
    uint32_t rows;          // tokens * Hkv (< 2^30)
    FastDiv div_h, div_n;   // by Hkv, by n_new (unused with cu_rows)
    int32_t lg_p;           // log2 page_size
    int32_t lg_lanes_k, lg_lanes_v;  // log2 of group_k / 8 and group_v / 8 (lanes of 8 values per group)
    BlockLayout L;
};
cudaError_t launch_quantize_append(const QuantizeArgs& a, cudaStream_t stream);

struct DequantArgs {
    const uint8_t* pool;
    const int32_t* block_table;
    void* out_k;
    void* out_v;
    uint32_t* status;
    int32_t max_blocks, b, start, n, Hkv, num_pages, out_fp32;
    BlockLayout L;
};
cudaError_t launch_dequantize(const DequantArgs& a, cudaStream_t stream);

// Copy n16 16-byte words from src (device address of mapped pinned host memory) to dst on
// the device, as a kernel launched with programmatic dependent launch: it reads src while
// the kernel ahead of it on the stream finishes and writes dst only after that kernel has.
cudaError_t launch_stage_in(const void* src, void* dst, size_t n16, cudaStream_t stream);

// Decode attention: the persistent split-KV kernel with the split combine fused in.
struct DecodePlan {
    int32_t hk;           // kv heads per unit of work (4 when Hq == Hkv, Hkv % 4 == 0, P == 16; 2 for two
                          // slots per kv head in the weights and differential modes; else 1)
    int32_t hs;           // query-head slots per score thread: 1 (up to 4 per unit) or 2 (up to 8)
    int32_t ctas;         // CTAs of the persistent grid (4 warps each)
    int32_t stages;       // bulk-copy ring depth per warp, in units
    size_t smem_bytes;    // dynamic shared memory per CTA
    int32_t combine_warps; // warps per CTA of the combine kernel (one CTA per output row)
    size_t ws_pre_offset; // pages prefix per sequence, published by the decode grid
    size_t ws_ml_offset;  // (max, sum) of the warp partials
    size_t ws_o_offset;   // unnormalised outputs of the warp partials
    size_t ws_stat_offset;  // attention with weights: (max, 1 / sum) of each output row
    size_t ws_score_offset; // attention with weights: the scores of every attended position
    int32_t score_ld;       //   ... floats from one query head's scores to the next's
    size_t ws_bytes;      // total workspace bytes
};

// What a decode call computes besides, or instead of, plain attention.
enum class DecodeMode : int32_t {
    kPlain = 0,
    kWeights = 1,  // the positions' attention weights are added to an accumulator too
    kDiff = 2,     // the difference of two softmax maps (Hq counts virtual heads, two per query head)
};

struct DecodeArgs {
    const uint8_t* pool;
    const __half* q;
    const int32_t* block_table;
    const int32_t* seq_lens;
    float* out;
    uint8_t* workspace;
    int32_t max_blocks, B, Hq, Hkv, num_pages, max_len;
    float softmax_scale;
    BlockLayout L;
    // the decode step's fused append of one token per sequence (k_new == nullptr: none)
    const __half* k_new = nullptr;
    const __half* v_new = nullptr;
    const int32_t* append_pos = nullptr;
    uint8_t* pool_w = nullptr;
    // sliding window with sink tokens: the last `window` positions (0: all) and the first `sinks`
    int32_t window = 0;
    int32_t sinks = 0;
    // attention over the FP16 cache instead of the INT4 one (the comparison's baseline), or
    // (with int8 or wht also set) over the INT8 per-row cache or the rotated 4-bit cache;
    // all three take the CUDA-core kernel
    bool fp16 = false;
    bool int8 = false;
    bool wht = false;
    // attend seq_lens[b] - len_sub positions (the INT4 part of the mixed-precision decode)
    int32_t len_sub = 0;
    // status word (nullptr: the first word of the workspace)
    uint32_t* status = nullptr;
    // device address of mapped pinned host memory the combine also writes the output to
    // (the host-buffer decode step), or nullptr
    float* out_host = nullptr;
    // q (and the new rows) are written by the kernel just ahead on the stream, which lets
    // this grid start early: the grid reads q only after griddepcontrol.wait
    bool q_after_wait = false;
    // bound of the INT4 kernel's waits on copies in ns (0: the default, 250 ms), and the test
    // of that bound (each warp's, kWeights: each of the first CTA's, first page copy announced 16
    // bytes larger than it is)
    uint64_t wait_ns = 0;
    bool withhold_first_copy = false;
    DecodeMode mode = DecodeMode::kPlain;
    // kWeights: weights[b][kv head][t] = decay * weights + the sum over the kv head's query
    // heads of position t's softmax weight (decay 0: the sum alone); weights_ld floats per kv head
    float* weights = nullptr;
    int32_t weights_ld = 0;
    float decay = 1.f;
    // kWeights over INT8 pages of 64 tokens: half-page units; L.P and max_blocks then count halves,
    // page_ld is the block table's row and page_P the page's tokens (0: units are pages)
    int32_t page_ld = 0, page_P = 0;
    // kDiff: out = out_scale * norm(map 1 - lambda[query head] * map 2), norm an RMS norm over
    // head_dim with gain norm_weight and norm_eps (norm_weight nullptr: none)
    const float* lambda = nullptr;
    const float* norm_weight = nullptr;
    float norm_eps = 0.f;
    float out_scale = 1.f;
};

// The FP16 cache of the latency comparison: block (page, kv head) holds K rows P x d fp16,
// then V rows P x d fp16.
struct Fp16AppendArgs {
    uint8_t* pool16;
    const __half* k;
    const __half* v;
    const int32_t* block_table;
    const int32_t* start_pos;
    uint32_t* status;
    int32_t max_blocks, B, n_new, Hkv, d, P, num_pages;
};
struct Fp16DequantArgs {
    const uint8_t* pool;
    uint8_t* pool16;
    const int32_t* block_table;
    const int32_t* seq_lens;
    uint32_t* status;
    int32_t max_blocks, B, Hkv, num_pages;
    BlockLayout L;
};
cudaError_t launch_fp16_append(const Fp16AppendArgs& a, cudaStream_t stream);
// INT8 per-row cache: quantize-append, arguments as for the FP16 append
cudaError_t launch_int8_quantize_append(const Fp16AppendArgs& a, cudaStream_t stream);
cudaError_t launch_dequantize_to_fp16(const Fp16DequantArgs& a, long long max_pages, cudaStream_t stream);

// The rotated 4-bit codec (wht_codec.cu): its fp32 codebook (the 16 Lloyd-Max levels of
// the standard normal, ascending, and the 15 midpoints between them), computed once;
// quantize-append with the FP16 append's arguments (pool16 the codec's pool, d = 128);
// dequantization of positions [start, start + n) of sequence b to fp32 [n, Hkv, 128].
struct Wht4Codebook {
    float levels[16];
    float thresholds[15];
};
const Wht4Codebook& wht4_codebook();
cudaError_t launch_wht4_quantize_append(const Fp16AppendArgs& a, cudaStream_t stream);
cudaError_t launch_wht4_dequantize(const uint8_t* pool, const int32_t* block_table, int32_t max_blocks, int32_t b,
                                   int32_t start, int32_t n, float* out_k, float* out_v, uint32_t* status,
                                   int32_t Hkv, int32_t P, int32_t num_pages, cudaStream_t stream);

// Returns cudaErrorInvalidValue for a geometry no kernel instance covers.
cudaError_t plan_decode(const DecodeArgs& a, DecodePlan* plan);
cudaError_t launch_decode(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);
// the decode grid alone (its partials stay in the workspace), and the combine of two grids'
// partials (the mixed-precision decode)
cudaError_t launch_decode_grid(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);
cudaError_t launch_combine2(const DecodeArgs& a0, const DecodePlan& plan0, const DecodeArgs& a1,
                            const DecodePlan& plan1, cudaStream_t stream);

// Eviction from a cache (evict.cu).  Select: of each (sequence, kv head), the positions kept.
struct EvictSelectArgs {
    const float* weights;
    const int32_t* seq_lens;
    int32_t* kept;      // [B][Hkv][keep], ascending, -1 behind the kept ones
    int32_t* new_lens;  // [B]
    uint32_t* status;
    int32_t weights_ld, max_len, B, Hkv, keep, sinks, recent;
};
cudaError_t launch_evict_select(const EvictSelectArgs& a, cudaStream_t stream);

// Compact: the kept rows of each (sequence, kv head) to positions 0 .. of dst_table's pages.
// A block's row of a token is four pieces (K and V codes, K and V scales), piece i of
// row_bytes[i] bytes at sec_off[i] + slot * row_bytes[i].
struct EvictCompactArgs {
    uint8_t* pool;
    const int32_t* block_table;
    const int32_t* dst_table;
    const int32_t* seq_lens;
    const int32_t* kept;
    float* weights;     // or nullptr
    uint32_t* status;
    int32_t max_blocks, dst_max_blocks, weights_ld, B, Hkv, num_pages, keep, lg_p, block_bytes;
    int32_t sec_off[4], row_bytes[4];
};
cudaError_t launch_evict_compact(const EvictCompactArgs& a, cudaStream_t stream);

// ---- ragged batches of rows ------------------------------------------------------------------
// Rows cu_rows[b] .. cu_rows[b + 1] - 1 belong to sequence b; row cu_rows[b] + t of it is position
// start_pos[b] + t; rows from cu_rows[B] on belong to no sequence.

// Rotary positions and quantize-append (rope_append.cu).
struct RopeAppendArgs {
    uint8_t* pool;
    const __half* q;
    const __half* k;
    const __half* v;
    __half* q_out;
    const float* table;        // [table_len][rot]: rot / 2 cosines, then rot / 2 sines
    const int32_t* positions;  // [axes][rows], or nullptr (one axis): the row's position in the cache
    const int32_t* block_table;
    const int32_t* start_pos;
    const int32_t* cu_rows;
    uint32_t* status;
    long long q_stride, k_stride, v_stride, q_out_stride;  // values from one row to the next
    int32_t rows, B, Hq, Hkv, max_blocks, num_pages, lg_p, table_len;
    int32_t rot, inter, axes, bound0, bound1;  // pairs below bound0 turn with axis 0, below bound1 with axis 1
    int32_t slices;                            // parts of a row's heads, each a warp's (set by the launcher)
    BlockLayout L;
};
cudaError_t launch_rope_append(RopeAppendArgs a, cudaStream_t stream);

struct DequantRowsArgs {
    const uint8_t* pool;
    const int32_t* block_table;
    const int32_t* start_pos;
    const int32_t* cu_rows;
    void* out_k;
    void* out_v;
    uint32_t* status;
    int32_t rows, B, Hkv, max_blocks, num_pages, lg_p, out_fp32, slices;
    BlockLayout L;
};
cudaError_t launch_dequantize_rows(DequantRowsArgs a, cudaStream_t stream);

// Blocks of 8 warps for `tasks` rows, each in `slices` parts: as many parts (at most most_slices) as
// leave every warp of the device at most one.
int rows_grid(long long tasks, int most_slices, int warps_per_sm, int* slices);
// Launch with programmatic dependent launch (the kernel waits with griddepcontrol.wait).
cudaError_t launch_rows(const void* kernel, int blocks, int threads, void** args, cudaStream_t stream);

// A page of a latent cache: P rows of L / 2 bytes of codes, P rows of L / G fp16 scales, P rows of R
// fp16 rotary keys (every part a multiple of 16 bytes).
struct LatentLayout {
    int32_t L, R, P, G;
    int32_t scales, rope, bytes;  // offsets of the parts, bytes of a page
};
inline LatentLayout latent_layout(const kvq_latent_config& c) {
    LatentLayout l;
    l.L = c.latent_dim;
    l.R = c.rope_dim;
    l.P = c.page_size;
    l.G = c.group;
    l.scales = l.P * l.L / 2;
    l.rope = l.scales + l.P * (l.L / l.G) * 2;
    l.bytes = l.rope + l.P * l.R * 2;
    return l;
}

struct LatentAppendArgs {
    uint8_t* pool;
    const __half* x;  // [rows][L + R], rows x_stride values apart
    const float* gain;
    const __half* q_pe;  // [rows][H][R], rows q_pe_stride values apart, or nullptr
    __half* q_out;       // [rows][H][L + R]
    const float* table;
    const int32_t* positions;
    const int32_t* block_table;
    const int32_t* start_pos;
    const int32_t* cu_rows;
    uint32_t* status;
    long long x_stride, q_pe_stride;
    float eps;
    int32_t rows, B, H, max_blocks, num_pages, lg_p, table_len, inter, slices;
    LatentLayout lay;
};
cudaError_t launch_latent_append(LatentAppendArgs a, cudaStream_t stream);

struct LatentDequantArgs {
    const uint8_t* pool;
    const int32_t* block_table;
    const int32_t* start_pos;
    const int32_t* cu_rows;
    __half* out;
    uint32_t* status;
    int32_t rows, B, max_blocks, num_pages, lg_p;
    LatentLayout lay;
};
cudaError_t launch_latent_dequantize(LatentDequantArgs a, cudaStream_t stream);

// Attention of a ragged batch of query rows: row i of sequence b's n_b rows is position
// seq_lens[b] - n_b + i and attends to the positions up to its own.
struct ChunkArgs {
    const uint8_t* pool;
    const __half* q;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* cu_rows;
    __half* out;
    uint8_t* workspace;
    int32_t rows, B, Hq, Hkv, max_blocks, num_pages, lg_p, max_len;
    float softmax_scale;
    uint32_t wait_limit_ns = 0;  // not 0: a test of the bounded waits
    BlockLayout L;
};
// CTAs of the attention kernels on ragged batches: one per SM (0: no device).
int attention_ctas();
size_t chunk_workspace_bytes(const ChunkArgs& a);
cudaError_t launch_chunk_attention(const ChunkArgs& a, cudaStream_t stream);

struct LatentAttnArgs {
    const uint8_t* pool;
    const __half* q;  // [rows][H][L + R]
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* cu_rows;
    __half* out;  // [rows][H][L]
    uint8_t* workspace;
    int32_t rows, B, H, max_blocks, num_pages, lg_p, max_len;
    float softmax_scale;
    uint32_t wait_limit_ns = 0;  // not 0: a test of the bounded waits
    LatentLayout lay;
};
size_t latent_workspace_bytes(const LatentAttnArgs& a);
cudaError_t launch_latent_attention(const LatentAttnArgs& a, cudaStream_t stream);

}  // namespace kvq
