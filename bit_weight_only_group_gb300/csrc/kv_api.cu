// C-ABI entry points of the paged cache: host validation, then the kernels.
#include <cmath>

#include "qg_internal.h"

namespace qg {
namespace {

// What caches of either kind share: pages, heads, and the strides of the values, in units of `size` bytes.
qg_status check_pages(const void* k, const void* v, int num_pages, int page_size, int heads_kv, int head_dim,
                      int64_t page_stride, int64_t token_stride, int64_t head_stride, int size, const char* who)
{
    if (head_dim != 64 && head_dim != 128)
        return fail(QG_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128 (got %d)", who, head_dim);
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
        return fail(QG_ERR_UNSUPPORTED, "%s: page_size must be a power of two in 16..1024 (got %d)", who, page_size);
    if (num_pages < 1 || num_pages > (1 << 30))
        return fail(QG_ERR_INVALID_ARG, "%s: num_pages=%d not in 1..2^30", who, num_pages);
    if (heads_kv < 1 || heads_kv > 65536)
        return fail(QG_ERR_INVALID_ARG, "%s: heads_kv=%d not in 1..65536", who, heads_kv);
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(QG_ERR_ALIGNMENT, "%s: cache k and v must be 16-byte aligned", who);
    // a stride over one entry is never taken
    const struct { int64_t stride; int count; const char* name; } s[] = {
        {page_stride, num_pages, "page"}, {token_stride, page_size, "token"}, {head_stride, heads_kv, "head"}};
    for (const auto& e : s) {
        if (e.count == 1) continue;
        if (e.stride < head_dim || e.stride >= (int64_t)1 << 38)
            return fail(QG_ERR_INVALID_ARG, "%s: %s_stride=%lld not in head_dim..2^38", who, e.name, (long long)e.stride);
        if (e.stride * size % 16)
            return fail(QG_ERR_ALIGNMENT, "%s: %s_stride must be a multiple of %d elements", who, e.name, 16 / size);
    }
    return QG_OK;
}

qg_status check_cache(const qg_kv_cache* c, const char* who)
{
    if (!c) return fail(QG_ERR_INVALID_ARG, "%s: null cache", who);
    if (!c->k || !c->v) return fail(QG_ERR_INVALID_ARG, "%s: cache k or v is null", who);
    if (c->dtype != QG_T_BF16 && c->dtype != QG_T_F16)
        return fail(QG_ERR_UNSUPPORTED, "%s: cache dtype must be bf16 or fp16 (got %d)", who, c->dtype);
    return check_pages(c->k, c->v, c->num_pages, c->page_size, c->heads_kv, c->head_dim, c->page_stride, c->token_stride,
                       c->head_stride, 2, who);
}

qg_status check_cache(const qg_kv8_cache* c, const char* who)
{
    if (!c) return fail(QG_ERR_INVALID_ARG, "%s: null cache", who);
    if (!c->k || !c->v || !c->k_scale || !c->v_scale)
        return fail(QG_ERR_INVALID_ARG, "%s: cache k, v, k_scale or v_scale is null", who);
    const qg_status st = check_pages(c->k, c->v, c->num_pages, c->page_size, c->heads_kv, c->head_dim, c->page_stride,
                                     c->token_stride, c->head_stride, 1, who);
    if (st != QG_OK) return st;
    const struct { int64_t stride; int count; const char* name; } s[] = {
        {c->scale_page_stride, c->num_pages, "page"}, {c->scale_block_stride, c->page_size / QG_KV8_BLOCK, "block"},
        {c->scale_head_stride, c->heads_kv, "head"}};
    for (const auto& e : s)
        if (e.count > 1 && (e.stride < 1 || e.stride >= (int64_t)1 << 38))
            return fail(QG_ERR_INVALID_ARG, "%s: scale_%s_stride=%lld not in 1..2^38", who, e.name, (long long)e.stride);
    return QG_OK;
}

qg_status check_batch(int page_size, const qg_kv_batch* b, const char* who)
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
        if ((int64_t)b->table_ld * page_size < b->max_kv)
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

qg_status check_rope(const qg_rope* r, int head_dim, const char* who)
{
    if (!r) return QG_OK;
    if (!r->table) return fail(QG_ERR_INVALID_ARG, "%s: rope table is null", who);
    if (r->dim < 16 || r->dim % 16 || r->dim > head_dim)
        return fail(QG_ERR_UNSUPPORTED, "%s: rope dim must be a multiple of 16 in 16..head_dim (got %d)", who, r->dim);
    if (r->positions < 1) return fail(QG_ERR_INVALID_ARG, "%s: rope positions < 1", who);
    if (!aligned(r->table, 16) || !aligned(r->at, 4)) return fail(QG_ERR_ALIGNMENT, "%s: rope arrays misaligned", who);
    return QG_OK;
}

qg_status check_norm(const qg_head_norm* n, const char* who)
{
    if (!n || (!n->q && !n->k)) return QG_OK;
    if (n->dtype != QG_T_F32 && n->dtype != QG_T_BF16 && n->dtype != QG_T_F16)
        return fail(QG_ERR_INVALID_ARG, "%s: bad dtype %d of the norm weights", who, n->dtype);
    if (!(n->eps >= 0.0f) || !std::isfinite(n->eps)) return fail(QG_ERR_INVALID_ARG, "%s: eps must be finite and not negative", who);
    if (!aligned(n->q, 16) || !aligned(n->k, 16)) return fail(QG_ERR_ALIGNMENT, "%s: norm weights must be 16-byte aligned", who);
    return QG_OK;
}

// The arguments of appending that do not depend on the kind of cache; *nothing: there is nothing to do.
qg_status check_append(int page_size, int heads_kv, int head_dim, const qg_kv_batch* batch, const qg_head_norm* norm,
                       const qg_rope* rope, const void* q, int64_t ldq, int heads_q, const void* k, int64_t ldk,
                       const void* v, int64_t ldv, int xt, const void* q_out, int64_t ldq_out, bool* nothing,
                       const char* who)
{
    qg_status st = check_batch(page_size, batch, who);
    if (st != QG_OK) return st;
    if (xt != QG_T_F32 && xt != QG_T_BF16 && xt != QG_T_F16) return fail(QG_ERR_INVALID_ARG, "%s: bad xt %d", who, xt);
    if (heads_q < 0 || heads_q > 65536 * 128) return fail(QG_ERR_INVALID_ARG, "%s: heads_q=%d", who, heads_q);
    st = check_rope(rope, head_dim, who);
    if (st == QG_OK) st = check_norm(norm, who);
    if (st != QG_OK) return st;
    *nothing = batch->sequences == 0 || batch->tokens == 0;
    if (*nothing) return QG_OK;
    const int xs = xt == QG_T_F32 ? 4 : 2;
    const int64_t kv_width = (int64_t)heads_kv * head_dim, q_width = (int64_t)heads_q * head_dim;
    st = check_rows(k, ldk, kv_width, xs, "k", who);
    if (st == QG_OK) st = check_rows(v, ldv, kv_width, xs, "v", who);
    if (st == QG_OK && heads_q > 0) {
        st = check_rows(q, ldq, q_width, xs, "q", who);
        if (st == QG_OK) st = check_rows(q_out, ldq_out, q_width, 2, "q_out", who);
    }
    return st;
}

qg_status append(const char* who, const qg_kv_cache* cache, const qg_kv_batch* batch, const qg_head_norm* norm,
                 const qg_rope* rope, const void* q, int64_t ldq, int heads_q, const void* k, int64_t ldk, const void* v,
                 int64_t ldv, qg_dtype xt, void* q_out, int64_t ldq_out, void* stream)
{
    qg_status st = check_cache(cache, who);
    if (st != QG_OK) return st;
    bool nothing = false;
    st = check_append(cache->page_size, cache->heads_kv, cache->head_dim, batch, norm, rope, q, ldq, heads_q, k, ldk, v,
                      ldv, xt, q_out, ldq_out, &nothing, who);
    if (st != QG_OK || nothing) return st;
    return launch_kv_append(*cache, *batch, norm, rope, q, ldq, heads_q, k, ldk, v, ldv, xt, q_out, ldq_out,
                            static_cast<cudaStream_t>(stream));
}

template <typename Cache>
qg_status check_attn(const Cache* cache, const qg_kv_batch* batch, int heads_q, const char* who)
{
    qg_status st = check_cache(cache, who);
    if (st != QG_OK) return st;
    st = check_batch(cache->page_size, batch, who);
    if (st != QG_OK) return st;
    if (heads_q < 1 || heads_q % cache->heads_kv)
        return fail(QG_ERR_INVALID_ARG, "%s: heads_q=%d is not a multiple of heads_kv=%d", who, heads_q, cache->heads_kv);
    if ((int64_t)batch->prefix_len * cache->heads_kv > (int64_t)1 << 36)
        return fail(QG_ERR_UNSUPPORTED, "%s: more than 2^36 prefix keys over all heads", who);
    if ((int64_t)batch->tokens * heads_q > (int64_t)1 << 30)
        return fail(QG_ERR_UNSUPPORTED, "%s: more than 2^30 rows", who);
    return QG_OK;
}

// The arguments of attention beside cache, batch and heads, of a batch with work; need: of the workspace.
qg_status check_attn_arrays(const void* q, int64_t ldq, int64_t width, const void* out, int64_t ldo, int ot, const float* lse,
                            const void* ws, size_t ws_bytes, size_t need, const char* who)
{
    qg_status st = check_rows(q, ldq, width, 2, "q", who);
    if (st == QG_OK) st = check_rows(out, ldo, width, ot == QG_T_F32 ? 4 : 2, "out", who);
    if (st != QG_OK) return st;
    if (!aligned(lse, 4)) return fail(QG_ERR_ALIGNMENT, "%s: lse misaligned", who);
    if (need && (!ws || ws_bytes < need))
        return fail(QG_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", who, ws ? ws_bytes : (size_t)0, need);
    if (need && !aligned(ws, 256)) return fail(QG_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", who);
    return QG_OK;
}

qg_status check_scale(float scale, int ot, const char* who)
{
    if (ot != QG_T_F32 && ot != QG_T_BF16 && ot != QG_T_F16) return fail(QG_ERR_INVALID_ARG, "%s: bad ot %d", who, ot);
    if (!(scale > 0.0f) || !std::isfinite(scale * 1.4426950408889634f))
        return fail(QG_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
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
    return append("qkv_append", cache, batch, nullptr, rope, q, ldq, heads_q, k, ldk, v, ldv, xt, q_out, ldq_out, stream);
}

qg_status qkv_append_norm(const qg_kv_cache* cache, const qg_kv_batch* batch, const qg_head_norm* norm,
                          const qg_rope* rope, const void* q, int64_t ldq, int32_t heads_q, const void* k, int64_t ldk,
                          const void* v, int64_t ldv, qg_dtype xt, void* q_out, int64_t ldq_out, void* stream)
{
    return append("qkv_append_norm", cache, batch, norm, rope, q, ldq, heads_q, k, ldk, v, ldv, xt, q_out, ldq_out, stream);
}

qg_status qkv8_append(const qg_kv8_cache* cache, const qg_kv_batch* batch, const qg_head_norm* norm, const qg_rope* rope,
                      const void* q, int64_t ldq, int32_t heads_q, const void* k, int64_t ldk, const void* v, int64_t ldv,
                      qg_dtype xt, void* q_out, int64_t ldq_out, qg_dtype qt, void* stream)
{
    const char* who = "qkv8_append";
    qg_status st = check_cache(cache, who);
    if (st != QG_OK) return st;
    if (qt != QG_T_BF16 && qt != QG_T_F16) return fail(QG_ERR_INVALID_ARG, "%s: qt must be bf16 or fp16 (got %d)", who, (int)qt);
    bool nothing = false;
    st = check_append(cache->page_size, cache->heads_kv, cache->head_dim, batch, norm, rope, q, ldq, heads_q, k, ldk, v,
                      ldv, xt, q_out, ldq_out, &nothing, who);
    if (st != QG_OK || nothing) return st;
    return launch_kv8_append(*cache, *batch, norm, rope, q, ldq, heads_q, k, ldk, v, ldv, xt, q_out, ldq_out, qt,
                             static_cast<cudaStream_t>(stream));
}

qg_status qkv8_read(const qg_kv8_cache* cache, const qg_kv_batch* batch, void* k, int64_t ldk, void* v, int64_t ldv,
                    qg_dtype ot, void* stream)
{
    const char* who = "qkv8_read";
    qg_status st = check_cache(cache, who);
    if (st != QG_OK) return st;
    st = check_batch(cache->page_size, batch, who);
    if (st != QG_OK) return st;
    if (ot != QG_T_F32 && ot != QG_T_BF16 && ot != QG_T_F16) return fail(QG_ERR_INVALID_ARG, "%s: bad ot %d", who, (int)ot);
    if (batch->sequences == 0 || batch->tokens == 0) return QG_OK;
    const int64_t width = (int64_t)cache->heads_kv * cache->head_dim;
    st = check_rows(k, ldk, width, ot == QG_T_F32 ? 4 : 2, "k", who);
    if (st == QG_OK) st = check_rows(v, ldv, width, ot == QG_T_F32 ? 4 : 2, "v", who);
    if (st != QG_OK) return st;
    return launch_kv8_read(*cache, *batch, k, ldk, v, ldv, ot, static_cast<cudaStream_t>(stream));
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
    if (st == QG_OK) st = check_scale(scale, ot, who);
    if (st != QG_OK || batch->sequences == 0 || batch->tokens == 0) return st;
    st = check_attn_arrays(q, ldq, (int64_t)heads_q * cache->head_dim, out, ldo, ot, lse, ws, ws_bytes,
                           attn_workspace_bytes(*cache, *batch, heads_q), who);
    if (st != QG_OK) return st;
    return launch_attn(*cache, *batch, q, ldq, heads_q, scale, out, ldo, ot, lse, ws, static_cast<cudaStream_t>(stream));
}

qg_status qattn8_workspace_size(const qg_kv8_cache* cache, const qg_kv_batch* batch, int32_t heads_q, size_t* bytes)
{
    if (!bytes) return fail(QG_ERR_INVALID_ARG, "qattn8_workspace_size: bytes is null");
    qg_status st = check_attn(cache, batch, heads_q, "qattn8_workspace_size");
    if (st != QG_OK) return st;
    *bytes = batch->sequences == 0 || batch->tokens == 0 ? 0 : attn8_workspace_bytes(*cache, *batch, heads_q);
    return QG_OK;
}

qg_status qattn8_forward(const qg_kv8_cache* cache, const qg_kv_batch* batch, const void* q, int64_t ldq, int32_t heads_q,
                         qg_dtype qt, float scale, void* out, int64_t ldo, qg_dtype ot, float* lse, void* ws,
                         size_t ws_bytes, void* stream)
{
    const char* who = "qattn8_forward";
    qg_status st = check_attn(cache, batch, heads_q, who);
    if (st == QG_OK) st = check_scale(scale, ot, who);
    if (st != QG_OK) return st;
    if (qt != QG_T_BF16 && qt != QG_T_F16) return fail(QG_ERR_INVALID_ARG, "%s: qt must be bf16 or fp16 (got %d)", who, (int)qt);
    if (batch->sequences == 0 || batch->tokens == 0) return QG_OK;
    st = check_attn_arrays(q, ldq, (int64_t)heads_q * cache->head_dim, out, ldo, ot, lse, ws, ws_bytes,
                           attn8_workspace_bytes(*cache, *batch, heads_q), who);
    if (st != QG_OK) return st;
    return launch_attn8(*cache, *batch, q, ldq, heads_q, qt, scale, out, ldo, ot, lse, ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
