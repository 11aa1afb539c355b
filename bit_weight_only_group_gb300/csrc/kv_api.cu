// C-ABI entry points of the paged cache: host validation, then the kernels.
#include <cmath>

#include "qg_internal.h"

namespace qg {
namespace {

qg_status check_cache(const qg_kv_cache* c, const char* who)
{
    if (!c) return fail(QG_ERR_INVALID_ARG, "%s: null cache", who);
    if (!c->k || !c->v) return fail(QG_ERR_INVALID_ARG, "%s: cache k or v is null", who);
    if (c->dtype != QG_T_BF16 && c->dtype != QG_T_F16)
        return fail(QG_ERR_UNSUPPORTED, "%s: cache dtype must be bf16 or fp16 (got %d)", who, c->dtype);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(QG_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128 (got %d)", who, c->head_dim);
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return fail(QG_ERR_UNSUPPORTED, "%s: page_size must be a power of two in 16..1024 (got %d)", who, c->page_size);
    if (c->num_pages < 1 || c->num_pages > (1 << 30))
        return fail(QG_ERR_INVALID_ARG, "%s: num_pages=%d not in 1..2^30", who, c->num_pages);
    if (c->heads_kv < 1 || c->heads_kv > 65536)
        return fail(QG_ERR_INVALID_ARG, "%s: heads_kv=%d not in 1..65536", who, c->heads_kv);
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(QG_ERR_ALIGNMENT, "%s: cache k and v must be 16-byte aligned", who);
    // a stride over one entry is never taken
    const struct { int64_t stride; int count; const char* name; } s[] = {
        {c->page_stride, c->num_pages, "page"}, {c->token_stride, c->page_size, "token"}, {c->head_stride, c->heads_kv, "head"}};
    for (const auto& e : s) {
        if (e.count == 1) continue;
        if (e.stride < c->head_dim || e.stride >= (int64_t)1 << 38)
            return fail(QG_ERR_INVALID_ARG, "%s: %s_stride=%lld not in head_dim..2^38", who, e.name, (long long)e.stride);
        if (e.stride % 8) return fail(QG_ERR_ALIGNMENT, "%s: %s_stride must be a multiple of 8 elements", who, e.name);
    }
    return QG_OK;
}

qg_status check_batch(const qg_kv_cache& c, const qg_kv_batch* b, const char* who)
{
    if (!b) return fail(QG_ERR_INVALID_ARG, "%s: null batch", who);
    if (b->sequences < 0 || b->tokens < 0 || b->max_q < 0 || b->max_kv < 0 || b->prefix_len < 0 || b->table_ld < 0)
        return fail(QG_ERR_INVALID_ARG, "%s: negative size in the batch", who);
    if (b->sequences > 0 && b->tokens > 0) {
        if (!b->kv_len) return fail(QG_ERR_INVALID_ARG, "%s: kv_len is null", who);
        if (b->max_q < 1) return fail(QG_ERR_INVALID_ARG, "%s: max_q < 1", who);
        if (!b->cu_q && (b->tokens != b->sequences || b->max_q != 1))
            return fail(QG_ERR_INVALID_ARG, "%s: without cu_q, tokens must equal sequences and max_q be 1", who);
    }
    if (b->max_kv > 0) {
        if (!b->table) return fail(QG_ERR_INVALID_ARG, "%s: table is null", who);
        if ((int64_t)b->table_ld * c.page_size < b->max_kv)
            return fail(QG_ERR_INVALID_ARG, "%s: table_ld=%d pages hold fewer than max_kv=%d tokens", who, b->table_ld, b->max_kv);
    }
    if (b->prefix_len > 0 && !b->prefix_table) return fail(QG_ERR_INVALID_ARG, "%s: prefix_table is null", who);
    if ((int64_t)b->prefix_len + b->max_kv > (int64_t)1 << 30)
        return fail(QG_ERR_UNSUPPORTED, "%s: more than 2^30 keys a sequence", who);
    if (!aligned(b->table, 4) || !aligned(b->kv_len, 4) || !aligned(b->cu_q, 4) || !aligned(b->prefix_table, 4))
        return fail(QG_ERR_ALIGNMENT, "%s: table, kv_len, cu_q or prefix_table misaligned", who);
    return QG_OK;
}

// A [T, heads, head_dim] array with tokens ld elements of `size` bytes apart.
qg_status check_rows(const void* p, int64_t ld, int64_t width, int size, const char* name, const char* who)
{
    if (!p) return fail(QG_ERR_INVALID_ARG, "%s: %s is null", who, name);
    if (ld < width) return fail(QG_ERR_INVALID_ARG, "%s: ld of %s = %lld < %lld", who, name, (long long)ld, (long long)width);
    if (!aligned(p, 16) || ld * size % 16) return fail(QG_ERR_ALIGNMENT, "%s: %s must be 16-byte aligned, rows too", who, name);
    return QG_OK;
}

qg_status check_attn(const qg_kv_cache* cache, const qg_kv_batch* batch, int heads_q, const char* who)
{
    qg_status st = check_cache(cache, who);
    if (st != QG_OK) return st;
    st = check_batch(*cache, batch, who);
    if (st != QG_OK) return st;
    if (heads_q < 1 || heads_q % cache->heads_kv)
        return fail(QG_ERR_INVALID_ARG, "%s: heads_q=%d is not a multiple of heads_kv=%d", who, heads_q, cache->heads_kv);
    if ((int64_t)batch->prefix_len * cache->heads_kv > (int64_t)1 << 36)
        return fail(QG_ERR_UNSUPPORTED, "%s: more than 2^36 prefix keys over all heads", who);
    if ((int64_t)batch->tokens * heads_q > (int64_t)1 << 30)
        return fail(QG_ERR_UNSUPPORTED, "%s: more than 2^30 rows", who);
    return QG_OK;
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

qg_status qkv_append(const qg_kv_cache* cache, const qg_kv_batch* batch, const qg_rope* rope, const void* q, int64_t ldq,
                     int32_t heads_q, const void* k, int64_t ldk, const void* v, int64_t ldv, qg_dtype xt, void* q_out,
                     int64_t ldq_out, void* stream)
{
    const char* who = "qkv_append";
    qg_status st = check_cache(cache, who);
    if (st != QG_OK) return st;
    st = check_batch(*cache, batch, who);
    if (st != QG_OK) return st;
    if (xt != QG_T_F32 && xt != QG_T_BF16 && xt != QG_T_F16) return fail(QG_ERR_INVALID_ARG, "%s: bad xt %d", who, (int)xt);
    if (heads_q < 0 || heads_q > 65536 * 128) return fail(QG_ERR_INVALID_ARG, "%s: heads_q=%d", who, heads_q);
    if (rope) {
        if (!rope->table) return fail(QG_ERR_INVALID_ARG, "%s: rope table is null", who);
        if (rope->dim < 16 || rope->dim % 16 || rope->dim > cache->head_dim)
            return fail(QG_ERR_UNSUPPORTED, "%s: rope dim must be a multiple of 16 in 16..head_dim (got %d)", who, rope->dim);
        if (rope->positions < 1) return fail(QG_ERR_INVALID_ARG, "%s: rope positions < 1", who);
        if (!aligned(rope->table, 16) || !aligned(rope->at, 4)) return fail(QG_ERR_ALIGNMENT, "%s: rope arrays misaligned", who);
    }
    if (batch->sequences == 0 || batch->tokens == 0) return QG_OK;
    const int xs = xt == QG_T_F32 ? 4 : 2;
    const int64_t kv_width = (int64_t)cache->heads_kv * cache->head_dim;
    st = check_rows(k, ldk, kv_width, xs, "k", who);
    if (st == QG_OK) st = check_rows(v, ldv, kv_width, xs, "v", who);
    if (st == QG_OK && heads_q > 0) {
        st = check_rows(q, ldq, (int64_t)heads_q * cache->head_dim, xs, "q", who);
        if (st == QG_OK) st = check_rows(q_out, ldq_out, (int64_t)heads_q * cache->head_dim, 2, "q_out", who);
    }
    if (st != QG_OK) return st;
    return launch_kv_append(*cache, *batch, rope, q, ldq, heads_q, k, ldk, v, ldv, xt, q_out, ldq_out,
                            static_cast<cudaStream_t>(stream));
}

qg_status qattn_workspace_size(const qg_kv_cache* cache, const qg_kv_batch* batch, int32_t heads_q, size_t* bytes)
{
    if (!bytes) return fail(QG_ERR_INVALID_ARG, "qattn_workspace_size: bytes is null");
    qg_status st = check_attn(cache, batch, heads_q, "qattn_workspace_size");
    if (st != QG_OK) return st;
    *bytes = batch->sequences == 0 || batch->tokens == 0 ? 0 : attn_workspace_bytes(*cache, *batch, heads_q);
    return QG_OK;
}

qg_status qattn_forward(const qg_kv_cache* cache, const qg_kv_batch* batch, const void* q, int64_t ldq, int32_t heads_q,
                        float scale, void* out, int64_t ldo, qg_dtype ot, float* lse, void* ws, size_t ws_bytes,
                        void* stream)
{
    const char* who = "qattn_forward";
    qg_status st = check_attn(cache, batch, heads_q, who);
    if (st != QG_OK) return st;
    if (ot != QG_T_F32 && ot != QG_T_BF16 && ot != QG_T_F16) return fail(QG_ERR_INVALID_ARG, "%s: bad ot %d", who, (int)ot);
    if (!(scale > 0.0f) || !std::isfinite(scale * 1.4426950408889634f)) return fail(QG_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
    if (batch->sequences == 0 || batch->tokens == 0) return QG_OK;
    const int64_t width = (int64_t)heads_q * cache->head_dim;
    st = check_rows(q, ldq, width, 2, "q", who);
    if (st == QG_OK) st = check_rows(out, ldo, width, ot == QG_T_F32 ? 4 : 2, "out", who);
    if (st != QG_OK) return st;
    if (!aligned(lse, 4)) return fail(QG_ERR_ALIGNMENT, "%s: lse misaligned", who);
    const size_t need = attn_workspace_bytes(*cache, *batch, heads_q);
    if (need && (!ws || ws_bytes < need))
        return fail(QG_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", who, ws ? ws_bytes : (size_t)0, need);
    if (need && !aligned(ws, 256)) return fail(QG_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", who);
    return launch_attn(*cache, *batch, q, ldq, heads_q, scale, out, ldo, ot, lse, ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
