// Attention over the paged cache with a shared prefix: how a call is split,
// the kernel that joins the parts, and the page maps.
#include "attn.cuh"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

namespace qg {
namespace attn {
namespace {

constexpr int kTile = 64;     // keys of a tile of the row kernel
constexpr int kBlock = 128;   // keys of a block of the tile kernel

enum Path { kRows, kTiles };

// How a call is split.  Parts are numbered prefix first.
struct Plan {
    bool shared;                      // the prefix once for all rows, apart from the own tokens
    Path prefix_path, own_path;       // kernel of each (own_path: of prefix and own together when not shared)
    int prefix_parts, prefix_tiles;   // parts and tiles or blocks of one (shared)
    int own_parts, own_tiles;         // the same of the own tokens, or of prefix and own together
    int parts;                        // in all; 1: no joining, results are written at once
};

// Parts of `tiles` tiles for `units` independent units of work: enough for
// two CTAs on each SM, none below four tiles.
void split(int64_t units, int64_t tiles, int* parts, int* per)
{
    const int64_t want = std::max<int64_t>(1, ceil_div(2 * num_sms(), std::max<int64_t>(1, units)));
    const int64_t most = std::max<int64_t>(1, tiles / 4);
    const int64_t n = std::min(want, most);
    *per = (int)std::max<int64_t>(1, ceil_div(tiles, n));
    *parts = (int)std::max<int64_t>(1, ceil_div(tiles, *per));
}

// Parts of `blocks` blocks for `units` pairs of tiles on one CTA an SM: the
// count whose rounds of the whole card end soonest, an item costing its
// blocks and about three more to start and finish, and a part's results about
// a quarter block to write and to join.
void split_tiles(int64_t units, int64_t blocks, int* parts, int* per)
{
    const int64_t sms = num_sms();
    double best = 0;
    *parts = 1;
    *per = (int)std::max<int64_t>(1, blocks);
    for (int64_t n = 1; n <= 64 && n <= std::max<int64_t>(1, blocks / 2); n++) {
        const int64_t k = ceil_div(blocks, n);
        if (n > 1 && ceil_div(blocks, k) != n) continue;
        const int64_t rounds = ceil_div(units * n, sms);
        const double cost = (double)rounds * (k + 3) + (n > 1 ? 0.25 * n * ceil_div(units, sms) : 0.0);
        if (n == 1 || cost < best) {
            best = cost;
            *parts = (int)n;
            *per = (int)std::max<int64_t>(1, k);
        }
    }
}

Plan make_plan(const qg_kv_cache& c, const qg_kv_batch& b, int heads_q)
{
    Plan p{};
    const int64_t group = heads_q / c.heads_kv;
    const bool tiles = group <= 128;   // a tile holds whole tokens
    const int64_t per2 = 2 * std::max(1, tile_tokens(group));
    const int64_t own_units = (int64_t)b.sequences * c.heads_kv * ceil_div(group * b.max_q, 64);
    if (tiles && group * b.max_q > 64) {
        // rows enough for tiles within a sequence: prefix and own tokens in one pass, nothing to join
        p.own_path = kTiles;
        const int64_t pairs = std::min<int64_t>(b.tokens / per2 + b.sequences, b.sequences * ceil_div(b.max_q, per2));
        split_tiles(pairs * c.heads_kv, ceil_div(b.prefix_len, kBlock) + ceil_div(b.max_kv, kBlock), &p.own_parts, &p.own_tiles);
    } else if (b.sequences > 1 && b.prefix_len >= 256) {
        p.shared = true;
        p.own_path = kRows;
        if (tiles) {
            p.prefix_path = kTiles;
            split_tiles(ceil_div(b.tokens, per2) * c.heads_kv, ceil_div(b.prefix_len, kBlock), &p.prefix_parts, &p.prefix_tiles);
        } else {
            p.prefix_path = kRows;
            split(c.heads_kv * ceil_div(group * b.tokens, 64), ceil_div(b.prefix_len, kTile), &p.prefix_parts, &p.prefix_tiles);
        }
        split(own_units, ceil_div(b.max_kv, kTile), &p.own_parts, &p.own_tiles);
    } else {
        p.own_path = kRows;
        split(own_units, ceil_div(b.prefix_len, kTile) + ceil_div(b.max_kv, kTile), &p.own_parts, &p.own_tiles);
    }
    p.parts = p.prefix_parts + p.own_parts;
    return p;
}

size_t part_o_bytes(const Plan& p, int64_t rows, int dim)
{
    return p.parts > 1 ? align_up((size_t)p.parts * rows * dim * 4, 256) : 0;
}

// out[r] = sum_p w_p o_p / sum_p w_p l_p with w_p = 2^(m_p - max m), in the
// order of the parts: one warp a row, a lane 4 (or 2) of the row's values.
// Reads every part once: bound by L2, where the parts were just written.
template <int D>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ Args a, int parts)
{
    kv::pdl_wait();
    kv::pdl_release();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = (int)(row / a.heads_q), hq = (int)(row % a.heads_q);
    if (row >= a.rows || t >= kv::used_tokens(a.bt)) return;
    float m = -INFINITY, l = 0.0f;
    for (int p = lane; p < parts; p += 32) {
        const float2 v = __ldcg(a.part_ml + p * a.rows + row);
        if (v.y > 0.0f) m = fmaxf(m, v.x);
    }
#pragma unroll
    for (int i = 16; i > 0; i /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int base = 0; base < parts; base += 32) {
        float w = 0.0f, part_l = 0.0f;
        if (base + lane < parts) {
            const float2 v = __ldcg(a.part_ml + (base + lane) * a.rows + row);
            if (v.y > 0.0f) {
                w = exp2_approx(v.x - m);
                part_l = v.y * w;
            }
        }
        const int n = min(32, parts - base);
#pragma unroll 4
        for (int p = 0; p < n; p++) {
            const float wp = __shfl_sync(0xffffffffu, w, p);
            l += __shfl_sync(0xffffffffu, part_l, p);
            if (wp > 0.0f) {   // a part that saw nothing has no o
                const float* src = a.part_o + ((base + p) * a.rows + row) * D;
                if constexpr (D == 128) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(src) + lane);
                    o.x = fmaf(wp, v.x, o.x); o.y = fmaf(wp, v.y, o.y);
                    o.z = fmaf(wp, v.z, o.z); o.w = fmaf(wp, v.w, o.w);
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                    o.x = fmaf(wp, v.x, o.x); o.y = fmaf(wp, v.y, o.y);
                }
            }
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const long long at = t * a.ldo + (long long)hq * D;
    if constexpr (D == 128) store_out4(a, at + 4 * lane, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    else store_out2(a, at + 2 * lane, o.x * inv, o.y * inv);
    if (lane == 0) store_lse(a, row, m, l);
}

}  // namespace

cudaError_t launch_join(const Args& a, int parts, cudaStream_t s)
{
    const dim3 grid((unsigned)ceil_div(a.rows, 8));
    return a.c.dim == 128 ? kv::launch_dependent(k_attn_join<128>, grid, 256, 0, s, a, parts)
                          : kv::launch_dependent(k_attn_join<64>, grid, 256, 0, s, a, parts);
}

namespace {
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> encode{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode.load(std::memory_order_acquire);
    if (!fn) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f) return nullptr;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        encode.store(fn, std::memory_order_release);
    }
    return fn;
}

qg_status encode(CUtensorMap* map, int dtype, int rank, const void* base, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    if (!fn) return fail(QG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = fn(map, dtype == QG_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(QG_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return QG_OK;
}
}  // namespace

qg_status encode_pages(CUtensorMap* map, const qg_kv_cache& c, const void* base, int box_rows)
{
    // the stride of a dimension of one entry is never used: any valid one
    const cuuint64_t any = 16;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads_kv,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride * 2, c.heads_kv > 1 ? (cuuint64_t)c.head_stride * 2 : any,
                                   c.num_pages > 1 ? (cuuint64_t)c.page_stride * 2 : any};
    const cuuint32_t box[4] = {64u, (cuuint32_t)box_rows, 1u, 1u};
    return encode(map, c.dtype, 4, base, dims, strides, box);
}

qg_status encode_rows(CUtensorMap* map, int dtype, const void* q, int dim, int heads_q, int64_t ldq, int64_t tokens,
                      int group)
{
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads_q, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)ldq * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)group, (cuuint32_t)tile_tokens(group)};
    return encode(map, dtype, 3, q, dims, strides, box);
}

}  // namespace attn

size_t attn_workspace_bytes(const qg_kv_cache& cache, const qg_kv_batch& batch, int heads_q)
{
    const attn::Plan p = attn::make_plan(cache, batch, heads_q);
    const int64_t rows = (int64_t)batch.tokens * heads_q;
    if (p.parts <= 1) return 0;
    return attn::part_o_bytes(p, rows, cache.head_dim) + align_up((size_t)p.parts * rows * sizeof(float2), 256);
}

qg_status launch_attn(const qg_kv_cache& cache, const qg_kv_batch& batch, const void* q, int64_t ldq, int heads_q,
                      float scale, void* out, int64_t ldo, int ot, float* lse, void* ws, cudaStream_t s)
{
    const attn::Plan p = attn::make_plan(cache, batch, heads_q);
    attn::Args a;
    a.bt = kv::make_batch(batch);
    a.c = kv::make_cache(cache);
    a.q = q; a.ldq = ldq;
    a.heads_q = heads_q; a.group = heads_q / cache.heads_kv;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = out; a.ldo = ldo; a.out_type = ot; a.lse = lse;
    a.rows = (int64_t)batch.tokens * heads_q;
    a.part_o = p.parts > 1 ? static_cast<float*>(ws) : nullptr;
    a.part_ml = p.parts > 1 ? reinterpret_cast<float2*>(static_cast<char*>(ws) + attn::part_o_bytes(p, a.rows, cache.head_dim))
                            : nullptr;
    a.box_rows = std::min(cache.page_size, attn::kTile);
    a.status = device_status_ptr();
    CUtensorMap qmap, kmap, vmap;
    qg_status st = attn::encode_pages(&kmap, cache, cache.k, a.box_rows);
    if (st != QG_OK) return st;
    st = attn::encode_pages(&vmap, cache, cache.v, a.box_rows);
    if (st != QG_OK) return st;
    if (p.own_path == attn::kTiles || (p.shared && p.prefix_path == attn::kTiles)) {
        st = attn::encode_rows(&qmap, cache.dtype, q, cache.head_dim, heads_q, ldq, batch.tokens, a.group);
        if (st != QG_OK) return st;
    }
    cudaError_t e = cudaSuccess;
    if (p.shared)
        e = p.prefix_path == attn::kTiles
                ? attn::launch_tiles(a, cache.dtype, qmap, kmap, vmap, attn::kPrefix, 0, p.prefix_parts, p.prefix_tiles, s)
                : attn::launch_rows(a, cache.dtype, kmap, vmap, attn::kPrefix, 0, p.prefix_parts, p.prefix_tiles, s);
    const int keys = p.shared ? attn::kOwn : attn::kPrefix | attn::kOwn;
    if (e == cudaSuccess)
        e = p.own_path == attn::kTiles
                ? attn::launch_tiles(a, cache.dtype, qmap, kmap, vmap, keys, p.prefix_parts, p.own_parts, p.own_tiles, s)
                : attn::launch_rows(a, cache.dtype, kmap, vmap, keys, p.prefix_parts, p.own_parts, p.own_tiles, s);
    if (e == cudaSuccess && p.parts > 1) e = attn::launch_join(a, p.parts, s);
    if (e != cudaSuccess) return cuda_fail(e, "qattn_forward launch");
    return QG_OK;
}

}  // namespace qg
