// lq_attn_api.cu -- the C ABI of the softmax-attention operators (declared in
// include/lq.h): argument validation and dispatch.  Every entry point
// validates all of its arguments before it launches anything.  No exception
// crosses the ABI.
#include <cmath>
#include <cstdint>

#include "../../include/lq.h"
#include "lq_attn.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

lq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? LQ_OK : LQ_ERR_CUDA; }

lq_status check_config(const lq_attn_config *c) {
    if (!c) return LQ_ERR_INVALID_ARGUMENT;
    if (c->kv_heads < 1 || c->q_heads < 1 || c->q_heads > 4096 || c->q_heads % c->kv_heads != 0)
        return LQ_ERR_INVALID_ARGUMENT;
    if (c->head_dim < 1) return LQ_ERR_INVALID_ARGUMENT;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return LQ_ERR_UNSUPPORTED;
    if (c->io_dtype != LQ_F32 && c->io_dtype != LQ_BF16) return LQ_ERR_INVALID_ARGUMENT;
    if (c->norm != LQ_NORM_NONE && c->norm != LQ_NORM_L2 && c->norm != LQ_NORM_RMS)
        return LQ_ERR_INVALID_ARGUMENT;
    if (c->norm != LQ_NORM_NONE && !(c->eps >= 1e-30f && std::isfinite(c->eps))) return LQ_ERR_INVALID_ARGUMENT;
    if (c->rot_dim < 0 || c->rot_dim > c->head_dim || c->rot_dim % 16 != 0) return LQ_ERR_INVALID_ARGUMENT;
    if (c->rot_pairs != LQ_ROT_HALVES && c->rot_pairs != LQ_ROT_ADJACENT) return LQ_ERR_INVALID_ARGUMENT;
    if (c->window < 0) return LQ_ERR_INVALID_ARGUMENT;
    if (!(std::fabs(c->scale) <= 1e6f)) return LQ_ERR_INVALID_ARGUMENT;
    if (c->softcap != 0.0f && !(c->softcap >= 1e-3f && c->softcap <= 1e6f)) return LQ_ERR_INVALID_ARGUMENT;
    return LQ_OK;
}

lq_status check_cache(const lq_attn_config *c, const lq_kv_cache *k) {
    if (!k || !k->k_pages || !k->v_pages || !k->block_table) return LQ_ERR_INVALID_ARGUMENT;
    if (k->batch < 1 || k->num_pages < 1 || k->page_size < 1 || k->max_pages < 1) return LQ_ERR_INVALID_ARGUMENT;
    if ((int64_t)k->num_pages * c->kv_heads >= (1LL << 31) ||
        (int64_t)k->max_pages * k->page_size >= (1LL << 30))
        return LQ_ERR_INVALID_ARGUMENT;
    if (k->batch > lq::kMaxAttnBatch) return LQ_ERR_UNSUPPORTED;
    if (k->page_size < 16 || k->page_size > 256 || (k->page_size & (k->page_size - 1)) != 0)
        return LQ_ERR_UNSUPPORTED;
    if (!aligned16(k->k_pages) || !aligned16(k->v_pages) || !aligned4(k->block_table)) return LQ_ERR_MISALIGNED;
    return LQ_OK;
}

int page_shift(const lq_kv_cache *k) {
    int s = 0;
    while ((1 << s) < k->page_size) ++s;
    return s;
}

// A token-strided [tokens, heads, D] input.
lq_status check_rows(const lq_attn_config *c, const void *x, int64_t stride, int heads) {
    if (!x) return LQ_ERR_INVALID_ARGUMENT;
    const int64_t es = c->io_dtype == LQ_BF16 ? 2 : 4;
    if (stride < (int64_t)heads * c->head_dim || stride >= (1LL << 40)) return LQ_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || stride * es % 16 != 0) return LQ_ERR_MISALIGNED;
    return LQ_OK;
}

lq_status check_weights(const lq_attn_config *c, const float *qw, const float *kw, const float *cos_sin,
                        int32_t table_len) {
    if (c->norm == LQ_NORM_NONE && (qw || kw)) return LQ_ERR_INVALID_ARGUMENT;
    if ((c->rot_dim > 0) != (cos_sin != nullptr)) return LQ_ERR_INVALID_ARGUMENT;
    if (cos_sin && table_len < 1) return LQ_ERR_INVALID_ARGUMENT;
    if (!aligned16(qw) || !aligned16(kw) || !aligned16(cos_sin)) return LQ_ERR_MISALIGNED;
    return LQ_OK;
}

// cu_tokens / tokens of the ragged calls.
lq_status check_tokens(const lq_kv_cache *k, const int32_t *pos, const int32_t *cu, int32_t tokens) {
    if (!pos || tokens < 0) return LQ_ERR_INVALID_ARGUMENT;
    if (!cu && tokens % k->batch != 0) return LQ_ERR_INVALID_ARGUMENT;
    if (!aligned4(pos) || !aligned4(cu)) return LQ_ERR_MISALIGNED;
    return LQ_OK;
}

lq::RowsArgs rows_args(const lq_attn_config *c) {
    lq::RowsArgs a{};
    a.Hkv = c->kv_heads;
    a.norm = c->norm;
    a.rot = c->rot_dim;
    a.eps = c->eps;
    return a;
}

lq_status rows_launch(const lq_attn_config *c, const lq::RowsArgs &a, bool append, lq_stream_t stream) {
    return cuda_status(lq::launch_rows(a, c->head_dim, c->io_dtype == LQ_BF16, c->rot_pairs == LQ_ROT_ADJACENT,
                                       append, (cudaStream_t)stream));
}

lq::AttnArgs attn_args(const lq_attn_config *c, const lq_kv_cache *k, const int32_t *pos, const void *q, void *o) {
    lq::AttnArgs a{};
    a.k_pages = k->k_pages;
    a.v_pages = k->v_pages;
    a.block_table = k->block_table;
    a.pos = pos;
    a.q = q;
    a.o = o;
    a.B = k->batch;
    a.Hq = c->q_heads;
    a.Hkv = c->kv_heads;
    a.num_pages = k->num_pages;
    a.page_size = k->page_size;
    a.page_shift = page_shift(k);
    a.max_pages = k->max_pages;
    a.window = c->window;
    a.scale = c->scale;
    a.softcap = c->softcap;
    return a;
}

}  // namespace

extern "C" {

lq_status lq_qk_norm_rotate(const lq_attn_config *cfg, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, const float *q_weight, const float *k_weight,
                            const int32_t *positions, const float *cos_sin, int32_t table_len, int32_t tokens,
                            void *q_out, void *k_out, lq_stream_t stream) {
    lq_status e = check_config(cfg);
    if (e != LQ_OK) return e;
    if (tokens < 0) return LQ_ERR_INVALID_ARGUMENT;
    if (tokens == 0) return LQ_OK;
    e = check_rows(cfg, q, q_stride, cfg->q_heads);
    if (e != LQ_OK) return e;
    if ((k != nullptr) != (k_out != nullptr)) return LQ_ERR_INVALID_ARGUMENT;
    if (k) {
        e = check_rows(cfg, k, k_stride, cfg->kv_heads);
        if (e != LQ_OK) return e;
    }
    e = check_weights(cfg, q_weight, k_weight, cos_sin, table_len);
    if (e != LQ_OK) return e;
    if (!q_out || (cfg->rot_dim > 0 && !positions)) return LQ_ERR_INVALID_ARGUMENT;
    if (!aligned16(q_out) || !aligned16(k_out) || !aligned4(positions)) return LQ_ERR_MISALIGNED;
    lq::RowsArgs a = rows_args(cfg);
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.table_len = table_len;
    a.tokens = tokens;
    a.Hq = cfg->q_heads;
    if (!k) a.Hkv = 0;
    a.q_out = q_out;
    a.k_out = k_out;
    return rows_launch(cfg, a, false, stream);
}

lq_status lq_kv_append(const lq_attn_config *cfg, const lq_kv_cache *cache, const int32_t *pos,
                       const int32_t *cu_tokens, int32_t tokens, const void *q, int64_t q_stride, const void *k,
                       int64_t k_stride, const void *v, int64_t v_stride, const float *q_weight,
                       const float *k_weight, const float *cos_sin, int32_t table_len, void *q_out,
                       lq_stream_t stream) {
    lq_status e = check_config(cfg);
    if (e != LQ_OK) return e;
    e = check_cache(cfg, cache);
    if (e != LQ_OK) return e;
    e = check_tokens(cache, pos, cu_tokens, tokens);
    if (e != LQ_OK) return e;
    if (tokens == 0) return LQ_OK;
    if ((q != nullptr) != (q_out != nullptr)) return LQ_ERR_INVALID_ARGUMENT;
    if (q) {
        e = check_rows(cfg, q, q_stride, cfg->q_heads);
        if (e != LQ_OK) return e;
    }
    e = check_rows(cfg, k, k_stride, cfg->kv_heads);
    if (e != LQ_OK) return e;
    e = check_rows(cfg, v, v_stride, cfg->kv_heads);
    if (e != LQ_OK) return e;
    e = check_weights(cfg, q_weight, k_weight, cos_sin, table_len);
    if (e != LQ_OK) return e;
    if (!aligned16(q_out)) return LQ_ERR_MISALIGNED;
    lq::RowsArgs a = rows_args(cfg);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos_sin = cos_sin;
    a.table_len = table_len;
    a.tokens = tokens;
    a.Hq = q ? cfg->q_heads : 0;
    a.q_out = q_out;
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.block_table = cache->block_table;
    a.pos = pos;
    a.cu = cu_tokens;
    a.B = cache->batch;
    a.num_pages = cache->num_pages;
    a.page_size = cache->page_size;
    a.page_shift = page_shift(cache);
    a.max_pages = cache->max_pages;
    return rows_launch(cfg, a, true, stream);
}

int64_t lq_attn_workspace_bytes(const lq_attn_config *cfg, int32_t batch) {
    if (check_config(cfg) != LQ_OK || batch < 1 || batch > lq::kMaxAttnBatch) return -1;
    cudaError_t e = cudaSuccess;
    const size_t n = lq::attn_decode_workspace_bytes(batch, cfg->q_heads, cfg->kv_heads, cfg->head_dim,
                                                     cfg->io_dtype == LQ_BF16, &e);
    return e == cudaSuccess ? (int64_t)n : -1;
}

lq_status lq_attn_decode(const lq_attn_config *cfg, const lq_kv_cache *cache, const int32_t *pos, const void *q,
                         void *o, void *workspace, size_t workspace_bytes, lq_stream_t stream) {
    lq_status e = check_config(cfg);
    if (e != LQ_OK) return e;
    e = check_cache(cfg, cache);
    if (e != LQ_OK) return e;
    if (!pos || !q || !o || !workspace) return LQ_ERR_INVALID_ARGUMENT;
    if (!aligned4(pos) || !aligned16(q) || !aligned16(o) || !aligned16(workspace)) return LQ_ERR_MISALIGNED;
    // the line of tiles is counted in 32 bits
    const int64_t reach = (int64_t)cache->batch * cache->max_pages * cache->page_size;
    if (reach >= (1LL << 34) || reach * cfg->q_heads >= (1LL << 40)) return LQ_ERR_UNSUPPORTED;
    cudaError_t ce = cudaSuccess;
    const size_t need = lq::attn_decode_workspace_bytes(cache->batch, cfg->q_heads, cfg->kv_heads, cfg->head_dim,
                                                        cfg->io_dtype == LQ_BF16, &ce);
    if (ce != cudaSuccess) return LQ_ERR_CUDA;
    if (workspace_bytes < need) return LQ_ERR_INVALID_ARGUMENT;
    lq::AttnArgs a = attn_args(cfg, cache, pos, q, o);
    a.ws = static_cast<unsigned char *>(workspace);
    return cuda_status(lq::launch_attn_decode(a, cfg->head_dim, cfg->io_dtype == LQ_BF16, (cudaStream_t)stream));
}

lq_status lq_attn_prefill(const lq_attn_config *cfg, const lq_kv_cache *cache, const int32_t *pos,
                          const int32_t *cu_tokens, int32_t tokens, const void *q, void *o, lq_stream_t stream) {
    lq_status e = check_config(cfg);
    if (e != LQ_OK) return e;
    e = check_cache(cfg, cache);
    if (e != LQ_OK) return e;
    e = check_tokens(cache, pos, cu_tokens, tokens);
    if (e != LQ_OK) return e;
    if (tokens == 0) return LQ_OK;
    if (!q || !o) return LQ_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(o)) return LQ_ERR_MISALIGNED;
    lq::AttnArgs a = attn_args(cfg, cache, pos, q, o);
    a.cu = cu_tokens;
    a.tokens = tokens;
    return cuda_status(lq::launch_attn_prefill(a, cfg->head_dim, cfg->io_dtype == LQ_BF16, (cudaStream_t)stream));
}

}  // extern "C"
