// kvq_api_rows.cu -- the extern "C" boundary of the calls on ragged batches of rows: rotary append,
// read-back, chunk attention and the latent cache.  Argument checks and dispatch only.
#include <cmath>

#include "kvq.h"
#include "kvq_api.h"
#include "kvq_internal.h"

namespace {

using kvq::aligned;
using kvq::check_cfg;
using kvq::cuda_fail;
using kvq::fail;
using kvq::is_pow2_in;
using kvq::ok;

constexpr int32_t kMaxRows = 1 << 28;  // rows of a call, heads included below 2^31
constexpr int32_t kMaxLen = 1 << 30;   // positions of a sequence (32-bit position arithmetic)
constexpr int32_t kMaxBatch = 65536;

int lg(int32_t page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : 6; }

int check_rope(const kvq_rope_config* r, int32_t most) {
    if (!r) return fail(KVQ_EINVAL, "rope is NULL");
    if (!is_pow2_in(r->rotary_dim, 32, 256) || r->rotary_dim > most)
        return fail(KVQ_EUNSUPPORTED, "rotary_dim %d not in {32, 64, 128, 256} or > %d", r->rotary_dim, most);
    if (r->interleaved != 0 && r->interleaved != 1)
        return fail(KVQ_EINVAL, "interleaved %d is neither 0 nor 1", r->interleaved);
    if (r->axes < 1 || r->axes > 3) return fail(KVQ_EINVAL, "axes %d not in 1 .. 3", r->axes);
    if (r->axes > 1) {
        int64_t sum = 0;
        for (int i = 0; i < r->axes; ++i) {
            if (r->sections[i] < 0) return fail(KVQ_EINVAL, "sections[%d] = %d negative", i, r->sections[i]);
            sum += r->sections[i];
        }
        if (sum != r->rotary_dim / 2)
            return fail(KVQ_EINVAL, "sections add up to %lld pairs, not rotary_dim / 2 = %d", static_cast<long long>(sum),
                        r->rotary_dim / 2);
    }
    return KVQ_OK;
}

int check_latent(const kvq_latent_config* c) {
    if (!c) return fail(KVQ_EINVAL, "cfg is NULL");
    if (c->num_pages < 1) return fail(KVQ_EINVAL, "num_pages %d < 1", c->num_pages);
    if (c->latent_dim != 256 && c->latent_dim != 512)
        return fail(KVQ_EUNSUPPORTED, "latent_dim %d not in {256, 512}", c->latent_dim);
    if (c->rope_dim != 64) return fail(KVQ_EUNSUPPORTED, "rope_dim %d is not 64", c->rope_dim);
    if (!is_pow2_in(c->page_size, 16, 64)) return fail(KVQ_EUNSUPPORTED, "page_size %d not in {16, 32, 64}", c->page_size);
    if (!is_pow2_in(c->group, 32, 128)) return fail(KVQ_EUNSUPPORTED, "group %d not in {32, 64, 128}", c->group);
    if (static_cast<size_t>(c->num_pages) * kvq::latent_layout(*c).bytes > (static_cast<size_t>(1) << 46))
        return fail(KVQ_EINVAL, "pool larger than 64 TiB");
    return KVQ_OK;
}

// What every call on a ragged batch checks; *none where there is nothing to do.
int check_rows(int32_t batch, int32_t total_rows, int32_t heads, bool* none) {
    *none = false;
    if (batch < 0 || total_rows < 0) return fail(KVQ_EINVAL, "batch %d / total_rows %d negative", batch, total_rows);
    if (batch > kMaxBatch) return fail(KVQ_EUNSUPPORTED, "batch %d > %d", batch, kMaxBatch);
    if (total_rows > kMaxRows || static_cast<int64_t>(total_rows) * heads >= (int64_t{1} << 31))
        return fail(KVQ_EINVAL, "total_rows %d with %d heads: more than a call takes", total_rows, heads);
    *none = batch == 0 || total_rows == 0;
    return KVQ_OK;
}

int check_places(const void* pool, const int32_t* block_table, int32_t max_blocks, const int32_t* per_seq,
                 const int32_t* cu_rows, const uint32_t* status) {
    if (max_blocks < 1) return fail(KVQ_EINVAL, "max_blocks %d < 1", max_blocks);
    if (!pool || !block_table || !per_seq || !cu_rows) return fail(KVQ_EINVAL, "NULL device pointer");
    if (!aligned(pool, 16)) return fail(KVQ_EINVAL, "pool must be 16-byte aligned");
    if (!aligned(block_table, 4) || !aligned(per_seq, 4) || !aligned(cu_rows, 4) || (status && !aligned(status, 4)))
        return fail(KVQ_EINVAL, "int32/uint32 arguments must be 4-byte aligned");
    return KVQ_OK;
}

// A matrix of fp16 rows `stride` values apart, `width` of them used.
int check_strided(const void* p, int64_t stride, int64_t width, const char* name) {
    if (!p) return fail(KVQ_EINVAL, "NULL device pointer (%s)", name);
    if (!aligned(p, 16)) return fail(KVQ_EINVAL, "%s must be 16-byte aligned", name);
    if (stride < width || stride % 8 || stride > (int64_t{1} << 31))
        return fail(KVQ_EINVAL, "%s: row stride %lld below %lld, above 2^31 or no multiple of 8", name,
                    static_cast<long long>(stride), static_cast<long long>(width));
    return KVQ_OK;
}

int check_table(const float* cos_sin, int32_t table_len, const int32_t* positions, int32_t axes) {
    if (!cos_sin || table_len < 1) return fail(KVQ_EINVAL, "no table of cosines and sines (table_len %d)", table_len);
    if (!aligned(cos_sin, 16)) return fail(KVQ_EINVAL, "cos_sin must be 16-byte aligned");
    if (axes > 1 && !positions) return fail(KVQ_EINVAL, "%d axes need positions", axes);
    if (positions && !aligned(positions, 4)) return fail(KVQ_EINVAL, "int32/uint32 arguments must be 4-byte aligned");
    return KVQ_OK;
}

int check_attention(const void* q, const void* out, int32_t max_len, float softmax_scale) {
    if (max_len < 0 || max_len > kMaxLen) return fail(KVQ_EINVAL, "max_len %d not in 0 .. 2^30", max_len);
    // (2^64: fp16 queries and keys then keep every score, in powers of two, below fp32's largest)
    if (!(std::fabs(softmax_scale) <= 1.8446744e19f)) return fail(KVQ_EINVAL, "softmax_scale is not finite or above 2^64");
    if (!q || !out) return fail(KVQ_EINVAL, "NULL device pointer");
    if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_EINVAL, "q and out must be 16-byte aligned");
    return KVQ_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (!workspace) return fail(KVQ_EINVAL, "NULL device pointer");
    if (!aligned(workspace, 256)) return fail(KVQ_EINVAL, "workspace must be 256-byte aligned");
    if (need == 0) return fail(KVQ_ECUDA, "no CUDA device");
    if (bytes < need) return fail(KVQ_EWORKSPACE, "workspace %zu bytes < %zu required", bytes, need);
    return KVQ_OK;
}

int check_chunk_shape(const kvq_cache_config* cfg, int32_t num_q_heads) {
    if (int e = check_cfg(cfg)) return e;
    if (num_q_heads < 1 || num_q_heads % cfg->num_kv_heads)
        return fail(KVQ_EINVAL, "num_q_heads %d not a multiple of num_kv_heads %d", num_q_heads, cfg->num_kv_heads);
    if (num_q_heads / cfg->num_kv_heads > 8)
        return fail(KVQ_EUNSUPPORTED, "query heads per KV head %d > 8", num_q_heads / cfg->num_kv_heads);
    if (cfg->head_dim == 256) return fail(KVQ_EUNSUPPORTED, "chunk attention supports head_dim 64 and 128");
    return KVQ_OK;
}

int check_latent_shape(const kvq_latent_config* cfg, int32_t num_heads) {
    if (int e = check_latent(cfg)) return e;
    if (num_heads < 1 || num_heads > 1024) return fail(KVQ_EINVAL, "num_heads %d not in 1 .. 1024", num_heads);
    return KVQ_OK;
}

int check_wait_limit(uint64_t ns) {
    if (ns < 1000 || ns > 10000000)
        return fail(KVQ_EINVAL, "wait_limit_ns %llu outside [1 us, 10 ms]", static_cast<unsigned long long>(ns));
    return KVQ_OK;
}

int chunk_attention_impl(const kvq_cache_config* cfg, const void* pool, const void* q, const int32_t* block_table,
                         int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_rows, int32_t batch,
                         int32_t total_rows, int32_t num_q_heads, int32_t max_len, float softmax_scale, void* out,
                         void* workspace, size_t workspace_bytes, kvq_stream_t stream, uint64_t wait_limit_ns = 0) {
    if (int e = check_chunk_shape(cfg, num_q_heads)) return e;
    bool none;
    if (int e = check_rows(batch, total_rows, num_q_heads, &none)) return e;
    if (none) return ok();
    if (int e = check_places(pool, block_table, max_blocks, seq_lens, cu_rows, nullptr)) return e;
    if (int e = check_attention(q, out, max_len, softmax_scale)) return e;
    kvq::ChunkArgs a{};
    a.pool = static_cast<const uint8_t*>(pool);
    a.q = static_cast<const __half*>(q);
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.cu_rows = cu_rows;
    a.out = static_cast<__half*>(out);
    a.workspace = static_cast<uint8_t*>(workspace);
    a.rows = total_rows;
    a.B = batch;
    a.Hq = num_q_heads;
    a.Hkv = cfg->num_kv_heads;
    a.max_blocks = max_blocks;
    a.num_pages = cfg->num_pages;
    a.lg_p = lg(cfg->page_size);
    a.max_len = max_len;
    a.softmax_scale = softmax_scale;
    a.wait_limit_ns = static_cast<uint32_t>(wait_limit_ns);
    a.L = kvq::block_layout(*cfg);
    if (int e = check_workspace(workspace, workspace_bytes, kvq::chunk_workspace_bytes(a))) return e;
    const cudaError_t e = kvq::launch_chunk_attention(a, reinterpret_cast<cudaStream_t>(stream));
    return e != cudaSuccess ? cuda_fail(e, "kvq_chunk_attention launch") : ok();
}

int latent_attention_impl(const kvq_latent_config* cfg, const void* pool, const void* q, const int32_t* block_table,
                          int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_rows, int32_t batch,
                          int32_t total_rows, int32_t num_heads, int32_t max_len, float softmax_scale, void* out,
                          void* workspace, size_t workspace_bytes, kvq_stream_t stream, uint64_t wait_limit_ns = 0) {
    if (int e = check_latent_shape(cfg, num_heads)) return e;
    bool none;
    if (int e = check_rows(batch, total_rows, num_heads, &none)) return e;
    if (none) return ok();
    if (int e = check_places(pool, block_table, max_blocks, seq_lens, cu_rows, nullptr)) return e;
    if (int e = check_attention(q, out, max_len, softmax_scale)) return e;
    kvq::LatentAttnArgs a{};
    a.pool = static_cast<const uint8_t*>(pool);
    a.q = static_cast<const __half*>(q);
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.cu_rows = cu_rows;
    a.out = static_cast<__half*>(out);
    a.workspace = static_cast<uint8_t*>(workspace);
    a.rows = total_rows;
    a.B = batch;
    a.H = num_heads;
    a.max_blocks = max_blocks;
    a.num_pages = cfg->num_pages;
    a.lg_p = lg(cfg->page_size);
    a.max_len = max_len;
    a.softmax_scale = softmax_scale;
    a.wait_limit_ns = static_cast<uint32_t>(wait_limit_ns);
    a.lay = kvq::latent_layout(*cfg);
    if (int e = check_workspace(workspace, workspace_bytes, kvq::latent_workspace_bytes(a))) return e;
    const cudaError_t e = kvq::launch_latent_attention(a, reinterpret_cast<cudaStream_t>(stream));
    return e != cudaSuccess ? cuda_fail(e, "kvq_latent_attention launch") : ok();
}

}  // namespace

extern "C" {

int kvq_rope_append(const kvq_cache_config* cfg, const kvq_rope_config* rope, void* pool, const void* q, int64_t q_stride,
                    const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* q_out, int64_t q_out_stride,
                    int32_t num_q_heads, const float* cos_sin, int32_t table_len, const int32_t* positions,
                    const int32_t* block_table, int32_t max_blocks, const int32_t* start_pos, const int32_t* cu_rows,
                    int32_t batch, int32_t total_rows, uint32_t* status, kvq_stream_t stream) {
    if (int e = check_cfg(cfg)) return e;
    if (int e = check_rope(rope, cfg->head_dim)) return e;
    if (num_q_heads < 0 || num_q_heads > 65536) return fail(KVQ_EINVAL, "num_q_heads %d not in 0 .. 65536", num_q_heads);
    bool none;
    if (cfg->num_kv_heads > 65536) return fail(KVQ_EUNSUPPORTED, "num_kv_heads %d > 65536", cfg->num_kv_heads);
    if (int e = check_rows(batch, total_rows, num_q_heads + 2 * cfg->num_kv_heads, &none)) return e;
    if (none) return ok();
    if (int e = check_places(pool, block_table, max_blocks, start_pos, cu_rows, status)) return e;
    const int64_t d = cfg->head_dim;
    if (num_q_heads > 0) {
        if (int e = check_strided(q, q_stride, num_q_heads * d, "q")) return e;
        if (int e = check_strided(q_out, q_out_stride, num_q_heads * d, "q_out")) return e;
        if (q == q_out && q_stride != q_out_stride) return fail(KVQ_EINVAL, "q_out is q, with another row stride");
    }
    if (int e = check_strided(k, k_stride, cfg->num_kv_heads * d, "k")) return e;
    if (int e = check_strided(v, v_stride, cfg->num_kv_heads * d, "v")) return e;
    if (int e = check_table(cos_sin, table_len, positions, rope->axes)) return e;
    kvq::RopeAppendArgs a{};
    a.pool = static_cast<uint8_t*>(pool);
    a.q = static_cast<const __half*>(q);
    a.k = static_cast<const __half*>(k);
    a.v = static_cast<const __half*>(v);
    a.q_out = static_cast<__half*>(q_out);
    a.table = cos_sin;
    a.positions = positions;
    a.block_table = block_table;
    a.start_pos = start_pos;
    a.cu_rows = cu_rows;
    a.status = status;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.rows = total_rows;
    a.B = batch;
    a.Hq = num_q_heads;
    a.Hkv = cfg->num_kv_heads;
    a.max_blocks = max_blocks;
    a.num_pages = cfg->num_pages;
    a.lg_p = lg(cfg->page_size);
    a.table_len = table_len;
    a.rot = rope->rotary_dim;
    a.inter = rope->interleaved;
    a.axes = rope->axes;
    a.bound0 = rope->axes > 1 ? rope->sections[0] : rope->rotary_dim / 2;
    a.bound1 = rope->axes > 1 ? rope->sections[0] + rope->sections[1] : rope->rotary_dim / 2;
    a.L = kvq::block_layout(*cfg);
    const cudaError_t e = kvq::launch_rope_append(a, reinterpret_cast<cudaStream_t>(stream));
    return e != cudaSuccess ? cuda_fail(e, "kvq_rope_append launch") : ok();
}

int kvq_dequantize_varlen(const kvq_cache_config* cfg, const void* pool, const int32_t* block_table, int32_t max_blocks,
                          const int32_t* start_pos, const int32_t* cu_rows, int32_t batch, int32_t total_rows,
                          void* out_k, void* out_v, int32_t out_dtype, uint32_t* status, kvq_stream_t stream) {
    if (int e = check_cfg(cfg)) return e;
    if (out_dtype != 0 && out_dtype != 1) return fail(KVQ_EINVAL, "out_dtype %d is neither 0 (fp16) nor 1 (fp32)", out_dtype);
    bool none;
    if (cfg->num_kv_heads > 65536) return fail(KVQ_EUNSUPPORTED, "num_kv_heads %d > 65536", cfg->num_kv_heads);
    if (int e = check_rows(batch, total_rows, cfg->num_kv_heads, &none)) return e;
    if (none) return ok();
    if (int e = check_places(pool, block_table, max_blocks, start_pos, cu_rows, status)) return e;
    if (!out_k || !out_v) return fail(KVQ_EINVAL, "NULL device pointer");
    if (!aligned(out_k, 16) || !aligned(out_v, 16)) return fail(KVQ_EINVAL, "out_k and out_v must be 16-byte aligned");
    kvq::DequantRowsArgs a{};
    a.pool = static_cast<const uint8_t*>(pool);
    a.block_table = block_table;
    a.start_pos = start_pos;
    a.cu_rows = cu_rows;
    a.out_k = out_k;
    a.out_v = out_v;
    a.status = status;
    a.rows = total_rows;
    a.B = batch;
    a.Hkv = cfg->num_kv_heads;
    a.max_blocks = max_blocks;
    a.num_pages = cfg->num_pages;
    a.lg_p = lg(cfg->page_size);
    a.out_fp32 = out_dtype;
    a.L = kvq::block_layout(*cfg);
    const cudaError_t e = kvq::launch_dequantize_rows(a, reinterpret_cast<cudaStream_t>(stream));
    return e != cudaSuccess ? cuda_fail(e, "kvq_dequantize_varlen launch") : ok();
}

size_t kvq_chunk_workspace_bytes(const kvq_cache_config* cfg, int32_t batch, int32_t num_q_heads, int32_t max_len) {
    if (check_chunk_shape(cfg, num_q_heads) != KVQ_OK) return 0;
    if (batch < 1 || batch > kMaxBatch || max_len < 0 || max_len > kMaxLen) {
        fail(KVQ_EINVAL, "batch %d, max_len %d", batch, max_len);
        return 0;
    }
    kvq::ChunkArgs a{};
    a.B = batch;
    a.Hq = num_q_heads;
    a.Hkv = cfg->num_kv_heads;
    a.max_len = max_len;
    a.L = kvq::block_layout(*cfg);
    const size_t n = kvq::chunk_workspace_bytes(a);
    if (n == 0) fail(KVQ_ECUDA, "no CUDA device");
    else ok();
    return n;
}

int kvq_chunk_attention(const kvq_cache_config* cfg, const void* pool, const void* q, const int32_t* block_table,
                        int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_rows, int32_t batch,
                        int32_t total_rows, int32_t num_q_heads, int32_t max_len, float softmax_scale, void* out,
                        void* workspace, size_t workspace_bytes, kvq_stream_t stream) {
    return chunk_attention_impl(cfg, pool, q, block_table, max_blocks, seq_lens, cu_rows, batch, total_rows, num_q_heads, max_len,
                                softmax_scale, out, workspace, workspace_bytes, stream);
}

int kvq_test_chunk_wait_timeout(const kvq_cache_config* cfg, const void* pool, const void* q, const int32_t* block_table,
                                int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_rows, int32_t batch,
                                int32_t total_rows, int32_t num_q_heads, int32_t max_len, float softmax_scale, void* out,
                                void* workspace, size_t workspace_bytes, uint64_t wait_limit_ns,
                                kvq_stream_t stream) {
    if (int e = check_wait_limit(wait_limit_ns)) return e;
    return chunk_attention_impl(cfg, pool, q, block_table, max_blocks, seq_lens, cu_rows, batch, total_rows, num_q_heads, max_len,
                                softmax_scale, out, workspace, workspace_bytes, stream, wait_limit_ns);
}

size_t kvq_latent_block_bytes(const kvq_latent_config* cfg) {
    if (check_latent(cfg) != KVQ_OK) return 0;
    return static_cast<size_t>(kvq::latent_layout(*cfg).bytes);
}

size_t kvq_latent_pool_bytes(const kvq_latent_config* cfg) {
    if (check_latent(cfg) != KVQ_OK) return 0;
    return static_cast<size_t>(cfg->num_pages) * kvq::latent_layout(*cfg).bytes;
}

int kvq_latent_append(const kvq_latent_config* cfg, const kvq_rope_config* rope, void* pool, const void* rows,
                      int64_t row_stride, const float* norm_weight, float norm_eps, const void* q_pe, int64_t q_pe_stride,
                      void* q_out, int32_t num_heads, const float* cos_sin, int32_t table_len, const int32_t* positions,
                      const int32_t* block_table, int32_t max_blocks, const int32_t* start_pos, const int32_t* cu_rows,
                      int32_t batch, int32_t total_rows, uint32_t* status, kvq_stream_t stream) {
    if (int e = check_latent(cfg)) return e;
    if (int e = check_rope(rope, cfg->rope_dim)) return e;
    if (rope->rotary_dim != cfg->rope_dim || rope->axes != 1)
        return fail(KVQ_EUNSUPPORTED, "a latent cache turns its whole rotary part with one axis");
    if (num_heads < 0 || num_heads > 1024) return fail(KVQ_EINVAL, "num_heads %d not in 0 .. 1024", num_heads);
    if (norm_weight && !(norm_eps >= 0.f && std::isfinite(norm_eps)))
        return fail(KVQ_EINVAL, "norm_eps is negative or not finite");
    bool none;
    if (int e = check_rows(batch, total_rows, num_heads > 0 ? num_heads : 1, &none)) return e;
    if (none) return ok();
    if (int e = check_places(pool, block_table, max_blocks, start_pos, cu_rows, status)) return e;
    if (int e = check_strided(rows, row_stride, cfg->latent_dim + cfg->rope_dim, "rows")) return e;
    if (norm_weight && !aligned(norm_weight, 16)) return fail(KVQ_EINVAL, "norm_weight must be 16-byte aligned");
    if (num_heads > 0) {
        if (int e = check_strided(q_pe, q_pe_stride, static_cast<int64_t>(num_heads) * cfg->rope_dim, "q_pe")) return e;
        if (!q_out) return fail(KVQ_EINVAL, "NULL device pointer (q_out)");
        if (!aligned(q_out, 16)) return fail(KVQ_EINVAL, "q_out must be 16-byte aligned");
    }
    if (int e = check_table(cos_sin, table_len, positions, 1)) return e;
    kvq::LatentAppendArgs a{};
    a.pool = static_cast<uint8_t*>(pool);
    a.x = static_cast<const __half*>(rows);
    a.gain = norm_weight;
    a.q_pe = num_heads > 0 ? static_cast<const __half*>(q_pe) : nullptr;
    a.q_out = static_cast<__half*>(q_out);
    a.table = cos_sin;
    a.positions = positions;
    a.block_table = block_table;
    a.start_pos = start_pos;
    a.cu_rows = cu_rows;
    a.status = status;
    a.x_stride = row_stride;
    a.q_pe_stride = q_pe_stride;
    a.eps = norm_eps;
    a.rows = total_rows;
    a.B = batch;
    a.H = num_heads;
    a.max_blocks = max_blocks;
    a.num_pages = cfg->num_pages;
    a.lg_p = lg(cfg->page_size);
    a.table_len = table_len;
    a.inter = rope->interleaved;
    a.lay = kvq::latent_layout(*cfg);
    const cudaError_t e = kvq::launch_latent_append(a, reinterpret_cast<cudaStream_t>(stream));
    return e != cudaSuccess ? cuda_fail(e, "kvq_latent_append launch") : ok();
}

int kvq_latent_dequantize(const kvq_latent_config* cfg, const void* pool, const int32_t* block_table, int32_t max_blocks,
                          const int32_t* start_pos, const int32_t* cu_rows, int32_t batch, int32_t total_rows, void* out,
                          uint32_t* status, kvq_stream_t stream) {
    if (int e = check_latent(cfg)) return e;
    bool none;
    if (int e = check_rows(batch, total_rows, 1, &none)) return e;
    if (none) return ok();
    if (int e = check_places(pool, block_table, max_blocks, start_pos, cu_rows, status)) return e;
    if (!out) return fail(KVQ_EINVAL, "NULL device pointer");
    if (!aligned(out, 16)) return fail(KVQ_EINVAL, "out must be 16-byte aligned");
    kvq::LatentDequantArgs a{};
    a.pool = static_cast<const uint8_t*>(pool);
    a.block_table = block_table;
    a.start_pos = start_pos;
    a.cu_rows = cu_rows;
    a.out = static_cast<__half*>(out);
    a.status = status;
    a.rows = total_rows;
    a.B = batch;
    a.max_blocks = max_blocks;
    a.num_pages = cfg->num_pages;
    a.lg_p = lg(cfg->page_size);
    a.lay = kvq::latent_layout(*cfg);
    const cudaError_t e = kvq::launch_latent_dequantize(a, reinterpret_cast<cudaStream_t>(stream));
    return e != cudaSuccess ? cuda_fail(e, "kvq_latent_dequantize launch") : ok();
}

size_t kvq_latent_workspace_bytes(const kvq_latent_config* cfg, int32_t batch, int32_t num_heads, int32_t max_len) {
    if (check_latent_shape(cfg, num_heads) != KVQ_OK) return 0;
    if (batch < 1 || batch > kMaxBatch || max_len < 0 || max_len > kMaxLen) {
        fail(KVQ_EINVAL, "batch %d, max_len %d", batch, max_len);
        return 0;
    }
    kvq::LatentAttnArgs a{};
    a.B = batch;
    a.H = num_heads;
    a.max_len = max_len;
    a.lay = kvq::latent_layout(*cfg);
    const size_t n = kvq::latent_workspace_bytes(a);
    if (n == 0) fail(KVQ_ECUDA, "no CUDA device");
    else ok();
    return n;
}

int kvq_latent_attention(const kvq_latent_config* cfg, const void* pool, const void* q, const int32_t* block_table,
                         int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_rows, int32_t batch,
                         int32_t total_rows, int32_t num_heads, int32_t max_len, float softmax_scale, void* out,
                         void* workspace, size_t workspace_bytes, kvq_stream_t stream) {
    return latent_attention_impl(cfg, pool, q, block_table, max_blocks, seq_lens, cu_rows, batch, total_rows, num_heads, max_len,
                                 softmax_scale, out, workspace, workspace_bytes, stream);
}

int kvq_test_latent_wait_timeout(const kvq_latent_config* cfg, const void* pool, const void* q, const int32_t* block_table,
                                 int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_rows, int32_t batch,
                                 int32_t total_rows, int32_t num_heads, int32_t max_len, float softmax_scale, void* out,
                                 void* workspace, size_t workspace_bytes, uint64_t wait_limit_ns,
                                 kvq_stream_t stream) {
    if (int e = check_wait_limit(wait_limit_ns)) return e;
    return latent_attention_impl(cfg, pool, q, block_table, max_blocks, seq_lens, cu_rows, batch, total_rows, num_heads, max_len,
                                 softmax_scale, out, workspace, workspace_bytes, stream, wait_limit_ns);
}

}  // extern "C"
