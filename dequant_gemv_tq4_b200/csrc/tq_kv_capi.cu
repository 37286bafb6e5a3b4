// tq_kv_capi.cu -- the extern "C" boundary of the key/value cache (include/tq.h):
// argument checks on the host, dispatch to the launchers.  No allocation.
#include "../../include/tq.h"
#include "tq_internal.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_dtype(tq_dtype d) { return d == TQ_F32 || d == TQ_BF16 || d == TQ_F16; }
size_t element_size(tq_dtype t) { return t == TQ_F32 ? 4 : 2; }
tq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA; }

// Head dimension, heads and page size of a cache; the positions of a sequence
// have to fit 31 bits.
tq_status check_cache_shape(int64_t heads, int64_t head_dim, int64_t page_size) {
    if (heads < 1 || head_dim < 1 || page_size < 1) return TQ_ERR_INVALID_ARG;
    if (heads > TQ_KV_MAX_HEADS || head_dim % 32 != 0 || head_dim > TQ_KV_MAX_HEAD_DIM) return TQ_ERR_SHAPE;
    if (page_size < 16 || page_size > TQ_KV_MAX_PAGE || (page_size & (page_size - 1)) != 0) return TQ_ERR_SHAPE;
    return TQ_OK;
}

tq_status check_cache(const tq_kv_cache *c, tq::KvCache *out) {
    if (!c) return TQ_ERR_INVALID_ARG;
    tq_status st = check_cache_shape(c->kv_heads, c->head_dim, c->page_size);
    if (st != TQ_OK) return st;
    if (c->pages < 0 || c->batch < 0 || c->pages_per_seq < 0 || c->page_table_ld < c->pages_per_seq)
        return TQ_ERR_INVALID_ARG;
    if (c->batch > TQ_KV_MAX_BATCH || c->pages > INT32_MAX) return TQ_ERR_SHAPE;
    // places fit 31 bits, and so do the groups of 16 tokens of all sequences
    if (c->pages_per_seq > ((int64_t)1 << 30) / c->page_size) return TQ_ERR_SHAPE;
    if (c->pages_per_seq * c->page_size > TQ_KV_MAX_CAPACITY / (c->batch > 0 ? c->batch : 1)) return TQ_ERR_SHAPE;
    if (c->pages > 0 && (!c->codes || !c->scales)) return TQ_ERR_INVALID_ARG;
    if (c->batch > 0 && c->pages_per_seq > 0 && !c->page_table) return TQ_ERR_INVALID_ARG;
    if (!aligned(c->codes, 16) || !aligned(c->scales, 16) || !aligned(c->page_table, 4)) return TQ_ERR_ALIGNMENT;
    out->codes = c->codes;
    out->scales = c->scales;
    out->page_table = c->page_table;
    out->pages = c->pages;
    out->table_ld = c->page_table_ld;
    out->batch = (int)c->batch;
    out->pages_per_seq = (int)c->pages_per_seq;
    out->kv_heads = c->kv_heads;
    out->head_dim = c->head_dim;
    out->page_shift = 0;
    while ((1 << out->page_shift) < c->page_size) ++out->page_shift;
    return TQ_OK;
}

// A [tokens][heads][dim] operand with unit element stride.
tq_status check_heads_operand(const void *p, int64_t token_stride, int64_t head_stride) {
    if (!p) return TQ_ERR_INVALID_ARG;
    if (token_stride < 0 || head_stride < 0) return TQ_ERR_INVALID_ARG;
    if (!aligned(p, 16) || token_stride % 8 != 0 || head_stride % 8 != 0) return TQ_ERR_ALIGNMENT;
    return TQ_OK;
}

tq_status check_rope(const float *inv_freq, int64_t rot, int64_t dim) {
    if (rot < 2 || rot % 2 != 0 || rot > dim) return TQ_ERR_SHAPE;
    if (!inv_freq) return TQ_ERR_INVALID_ARG;
    return aligned(inv_freq, 4) ? TQ_OK : TQ_ERR_ALIGNMENT;
}

// Sizes of an attention call (`heads` query heads over kv_heads).
tq_status check_attention_shape(int64_t batch, int64_t tree, int64_t heads, int64_t kv_heads, int64_t head_dim) {
    if (batch < 0 || tree < 0 || heads < 1) return TQ_ERR_INVALID_ARG;
    tq_status st = check_cache_shape(kv_heads, head_dim, 16);
    if (st != TQ_OK) return st;
    if (batch > TQ_KV_MAX_BATCH || tree > TQ_KV_MAX_TREE || heads > TQ_KV_MAX_HEADS || heads % kv_heads != 0)
        return TQ_ERR_SHAPE;
    return TQ_OK;
}

}  // namespace

extern "C" {

tq_status tq_rope(const void *x, void *out, tq_dtype t, int64_t tokens, int64_t heads, int64_t dim,
                  int64_t x_token_stride, int64_t x_head_stride, int64_t out_token_stride, int64_t out_head_stride,
                  const int32_t *positions, const tq_rope_desc *rope, void *stream) {
    if (tokens < 0 || heads < 0 || dim < 1 || !rope) return TQ_ERR_INVALID_ARG;
    if (tokens > TQ_KV_MAX_TOKENS || heads > TQ_KV_MAX_HEADS || dim > TQ_ROPE_MAX_DIM) return TQ_ERR_SHAPE;
    if (!valid_dtype(t)) return TQ_ERR_DTYPE;
    tq_status st = check_rope(rope->inv_freq, rope->rot_dim, dim);
    if (st != TQ_OK) return st;
    if (tokens == 0 || heads == 0) return TQ_OK;
    if (!x || !out || !positions) return TQ_ERR_INVALID_ARG;
    if (x_token_stride < 0 || x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0)
        return TQ_ERR_INVALID_ARG;
    if (!aligned(x, element_size(t)) || !aligned(out, element_size(t)) || !aligned(positions, 4))
        return TQ_ERR_ALIGNMENT;
    // in place only element for element
    if (x == out && ((tokens > 1 && x_token_stride != out_token_stride) ||
                     (heads > 1 && x_head_stride != out_head_stride)))
        return TQ_ERR_INVALID_ARG;
    tq::RopeJob j;
    j.x = x;
    j.out = out;
    j.positions = positions;
    j.inv_freq = rope->inv_freq;
    j.tokens = tokens;
    j.x_token = x_token_stride;
    j.x_head = x_head_stride;
    j.o_token = out_token_stride;
    j.o_head = out_head_stride;
    j.heads = (int)heads;
    j.dim = (int)dim;
    j.rot = rope->rot_dim;
    j.interleaved = rope->interleaved != 0;
    j.inverse = rope->inverse != 0;
    j.dtype = t;
    j.scale = rope->scale;
    return from_cuda(tq::launch_rope(j, (cudaStream_t)stream));
}

size_t tq_kv_codes_bytes(int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t page_size) {
    if (pages < 0 || pages > INT32_MAX || check_cache_shape(kv_heads, head_dim, page_size) != TQ_OK) return 0;
    return (size_t)pages * 2 * kv_heads * page_size * head_dim / 2;
}

size_t tq_kv_scales_bytes(int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t page_size) {
    return tq_kv_codes_bytes(pages, kv_heads, head_dim, page_size) / 4;
}

tq_status tq_kv_append(const tq_kv_cache *cache, const int32_t *seqs, const int32_t *places, int64_t tokens,
                       const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                       int64_t v_token_stride, int64_t v_head_stride, tq_dtype t, const int32_t *positions,
                       const tq_rope_desc *rope, void *stream) {
    tq::KvAppendJob j;
    tq_status st = check_cache(cache, &j.c);
    if (st != TQ_OK) return st;
    if (tokens < 0) return TQ_ERR_INVALID_ARG;
    if (tokens > TQ_KV_MAX_TOKENS) return TQ_ERR_SHAPE;
    if (!valid_dtype(t)) return TQ_ERR_DTYPE;
    if (rope) {
        if ((st = check_rope(rope->inv_freq, rope->rot_dim, cache->head_dim)) != TQ_OK) return st;
        if (rope->inverse) return TQ_ERR_UNSUPPORTED;
    }
    if (tokens == 0) return TQ_OK;
    if (!seqs || !places || (rope && !positions)) return TQ_ERR_INVALID_ARG;
    if (!aligned(seqs, 4) || !aligned(places, 4) || !aligned(positions, 4)) return TQ_ERR_ALIGNMENT;
    if ((st = check_heads_operand(k, k_token_stride, k_head_stride)) != TQ_OK) return st;
    if ((st = check_heads_operand(v, v_token_stride, v_head_stride)) != TQ_OK) return st;
    j.x[0] = k;
    j.x[1] = v;
    j.token_stride[0] = k_token_stride;
    j.token_stride[1] = v_token_stride;
    j.head_stride[0] = k_head_stride;
    j.head_stride[1] = v_head_stride;
    j.seqs = seqs;
    j.places = places;
    j.positions = rope ? positions : nullptr;
    j.inv_freq = rope ? rope->inv_freq : nullptr;
    j.rot = rope ? rope->rot_dim : 0;
    j.interleaved = rope ? rope->interleaved != 0 : 0;
    j.scale = rope ? rope->scale : 1.0f;
    j.tokens = tokens;
    j.dtype = t;
    return from_cuda(tq::launch_kv_append(j, (cudaStream_t)stream));
}

tq_status tq_kv_read(const tq_kv_cache *cache, const int32_t *seqs, const int32_t *places, int64_t tokens, void *k,
                     int64_t k_token_stride, int64_t k_head_stride, void *v, int64_t v_token_stride,
                     int64_t v_head_stride, tq_dtype t, void *stream) {
    tq::KvReadJob j;
    tq_status st = check_cache(cache, &j.c);
    if (st != TQ_OK) return st;
    if (tokens < 0) return TQ_ERR_INVALID_ARG;
    if (tokens > TQ_KV_MAX_TOKENS) return TQ_ERR_SHAPE;
    if (!valid_dtype(t)) return TQ_ERR_DTYPE;
    if (tokens == 0) return TQ_OK;
    if (!seqs || !places) return TQ_ERR_INVALID_ARG;
    if (!aligned(seqs, 4) || !aligned(places, 4)) return TQ_ERR_ALIGNMENT;
    if ((st = check_heads_operand(k, k_token_stride, k_head_stride)) != TQ_OK) return st;
    if ((st = check_heads_operand(v, v_token_stride, v_head_stride)) != TQ_OK) return st;
    j.out[0] = k;
    j.out[1] = v;
    j.token_stride[0] = k_token_stride;
    j.token_stride[1] = v_token_stride;
    j.head_stride[0] = k_head_stride;
    j.head_stride[1] = v_head_stride;
    j.seqs = seqs;
    j.places = places;
    j.tokens = tokens;
    j.dtype = t;
    return from_cuda(tq::launch_kv_read(j, (cudaStream_t)stream));
}

tq_status tq_kv_commit(const tq_kv_cache *cache, int64_t layers, int64_t code_layer_stride,
                       int64_t scale_layer_stride, const int32_t *lens, const int32_t *path, int64_t path_ld,
                       int64_t steps, void *stream) {
    tq::KvCommitJob j;
    tq_status st = check_cache(cache, &j.c);
    if (st != TQ_OK) return st;
    if (layers < 0 || steps < 0 || path_ld < steps) return TQ_ERR_INVALID_ARG;
    if (layers > TQ_KV_MAX_LAYERS || steps > TQ_KV_MAX_TREE) return TQ_ERR_SHAPE;
    if (layers > 1 && (code_layer_stride < 0 || scale_layer_stride < 0)) return TQ_ERR_INVALID_ARG;
    if (layers > 1 && (code_layer_stride % 16 != 0 || scale_layer_stride % 8 != 0)) return TQ_ERR_ALIGNMENT;
    // layers that share records would be moved more than once
    const size_t pool = tq_kv_codes_bytes(cache->pages, cache->kv_heads, cache->head_dim, cache->page_size);
    if (layers > 1 && ((size_t)code_layer_stride < pool || 2 * (size_t)scale_layer_stride < pool / 4))
        return TQ_ERR_INVALID_ARG;
    if (layers == 0 || steps == 0 || cache->batch == 0) return TQ_OK;
    if (!lens || !path) return TQ_ERR_INVALID_ARG;
    if (!aligned(lens, 4) || !aligned(path, 4)) return TQ_ERR_ALIGNMENT;
    j.layers = layers;
    j.code_layer = layers > 1 ? code_layer_stride : 0;
    j.scale_layer = layers > 1 ? scale_layer_stride : 0;
    j.lens = lens;
    j.path = path;
    j.path_ld = path_ld;
    j.steps = (int)steps;
    return from_cuda(tq::launch_kv_commit(j, (cudaStream_t)stream));
}

size_t tq_kv_attention_workspace_bytes(int64_t batch, int64_t tree, int64_t heads, int64_t kv_heads,
                                       int64_t head_dim) {
    tq::DeviceInfo di;
    if (check_attention_shape(batch, tree, heads, kv_heads, head_dim) != TQ_OK || tq::device_info(&di) != cudaSuccess)
        return 0;
    return tq::attention_workspace_bytes(batch, (int)tree, (int)heads, (int)kv_heads, (int)head_dim, di.sm_count);
}

tq_status tq_kv_attention(const tq_kv_cache *cache, const int32_t *lens, const int32_t *parents, int64_t parents_ld,
                          const void *q, tq_dtype qt, int64_t q_batch_stride, int64_t q_token_stride,
                          int64_t q_head_stride, void *out, tq_dtype ot, int64_t out_batch_stride,
                          int64_t out_token_stride, int64_t out_head_stride, int64_t tree, int64_t heads, float scale,
                          void *workspace, size_t ws_bytes, void *stream) {
    tq::AttentionJob j;
    tq_status st = check_cache(cache, &j.c);
    if (st != TQ_OK) return st;
    if ((st = check_attention_shape(cache->batch, tree, heads, cache->kv_heads, cache->head_dim)) != TQ_OK) return st;
    if (!valid_dtype(qt) || !valid_dtype(ot)) return TQ_ERR_DTYPE;
    if (cache->batch == 0 || tree == 0) return TQ_OK;
    if (cache->pages_per_seq < 1) return TQ_ERR_SHAPE;
    if (!lens || (parents && parents_ld < tree)) return TQ_ERR_INVALID_ARG;
    if (!aligned(lens, 4) || !aligned(parents, 4)) return TQ_ERR_ALIGNMENT;
    if (q_batch_stride < 0 || out_batch_stride < 0) return TQ_ERR_INVALID_ARG;
    if (q_batch_stride % 8 != 0 || out_batch_stride % 8 != 0) return TQ_ERR_ALIGNMENT;
    if ((st = check_heads_operand(q, q_token_stride, q_head_stride)) != TQ_OK) return st;
    if ((st = check_heads_operand(out, out_token_stride, out_head_stride)) != TQ_OK) return st;
    if (!(scale <= TQ_KV_MAX_SCALE && scale >= -TQ_KV_MAX_SCALE)) return TQ_ERR_INVALID_ARG;
    tq::DeviceInfo di;
    if (tq::device_info(&di) != cudaSuccess) return TQ_ERR_CUDA;
    if (!workspace || !aligned(workspace, 256) ||
        ws_bytes < tq::attention_workspace_bytes(cache->batch, (int)tree, (int)heads, cache->kv_heads,
                                                 cache->head_dim, di.sm_count))
        return TQ_ERR_WORKSPACE;
    j.lens = lens;
    j.parents = parents;
    j.parents_ld = parents_ld;
    j.q = q;
    j.q_batch = q_batch_stride;
    j.q_token = q_token_stride;
    j.q_head = q_head_stride;
    j.out = out;
    j.o_batch = out_batch_stride;
    j.o_token = out_token_stride;
    j.o_head = out_head_stride;
    j.tree = (int)tree;
    j.heads = (int)heads;
    j.qdtype = qt;
    j.odtype = ot;
    j.scale = scale;
    j.workspace = static_cast<char *>(workspace);
    return from_cuda(tq::launch_attention(j, di.sm_count, (cudaStream_t)stream));
}

}  // extern "C"
