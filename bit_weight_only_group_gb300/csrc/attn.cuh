// Declarations shared by the attention kernels: their arguments, the parts
// their partial results are kept in, and TMA loads of cache pages.
//
// A part is the attention of a row (one query head of one token) over some of
// its keys, kept as the running maximum m of scale * log2(e) * q.k, the sum l
// of 2^(s - m), and o = sum 2^(s - m) v.  Parts (m1, l1, o1), (m2, l2, o2)
// join to m = max, l = l1 2^(m1-m) + l2 2^(m2-m), o likewise; o / l is the
// attention over both.  All three are fp32.
#pragma once

#include <cuda.h>

#include "kv_batch.cuh"
#include "ptx.cuh"

namespace qg {
namespace attn {

using kv::Batch;
using kv::Cache;

struct Args {
    Batch bt;
    Cache c;
    const void* q;
    long long ldq;
    int heads_q, group;          // group = heads_q / heads_kv
    float scale_log2;            // scale * log2(e)
    void* out;
    long long ldo;
    int out_type;
    float* lse;                  // or null
    // partial results: o of part p, row r at part_o + (p * rows + r) * dim, (m, l) at part_ml + p * rows + r
    float* part_o;
    float2* part_ml;
    long long rows;              // T * heads_q
    int box_rows;                // key rows of one TMA box
    int* status;
};

constexpr float kLn2 = 0.69314718055994530942f;

// Values of a finished row, two or four at a time.
__device__ __forceinline__ void store_out2(const Args& a, long long at, float x, float y)
{
    if (a.out_type == QG_T_F32)
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(x, y);
    else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) =
            a.out_type == QG_T_BF16 ? kv::pack2<__nv_bfloat16>(x, y) : kv::pack2<__half>(x, y);
}
__device__ __forceinline__ void store_out4(const Args& a, long long at, float4 v)
{
    if (a.out_type == QG_T_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
    else if (a.out_type == QG_T_BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
            make_uint2(kv::pack2<__nv_bfloat16>(v.x, v.y), kv::pack2<__nv_bfloat16>(v.z, v.w));
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
            make_uint2(kv::pack2<__half>(v.x, v.y), kv::pack2<__half>(v.z, v.w));
}
__device__ __forceinline__ void store_lse(const Args& a, long long row, float m, float l)
{
    if (a.lse) a.lse[row] = l > 0.0f ? kLn2 * (m + log2f(l)) : -INFINITY;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// Page number of entry e of a table of n entries; num_pages (a box past the
// tensor, which TMA fills with zeros) where there is none to follow.
__device__ __forceinline__ int page_of(const Args& a, const int* table, int n, int e)
{
    const int p = e < n ? __ldg(table + e) : -1;
    if (p >= 0 && p < a.c.num_pages) return p;
    kv::report(a.status);
    return a.c.num_pages;
}

// Host side.
// Map of K or V pages: dimensions (dim, place, head, page), boxes of 64 values x box_rows places.
qg_status encode_pages(CUtensorMap* map, const qg_kv_cache& c, const void* base, int box_rows);
// Map of the query rows: dimensions (dim, head, token), boxes of 64 values x a group x a tile's tokens.
qg_status encode_rows(CUtensorMap* map, int dtype, const void* q, int dim, int heads_q, int64_t ldq, int64_t tokens,
                      int group);

// The kernels' launches.  A keys flag says what a row sees: the shared
// prefix, its own sequence's tokens, or both in that order.
enum Keys { kPrefix = 1, kOwn = 2 };
cudaError_t launch_rows(const Args& a, int dtype, const CUtensorMap& kmap, const CUtensorMap& vmap, int keys,
                        int part0, int parts, int tiles_per_part, cudaStream_t s);
// Tokens of a tile of the tile kernel (its rows: that times the group, at most 128).
inline int tile_tokens(int64_t group) { return (int)(128 / group); }
cudaError_t launch_tiles(const Args& a, int dtype, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, int keys, int part0, int parts, int blocks_per_part, cudaStream_t s);
cudaError_t launch_join(const Args& a, int parts, cudaStream_t s);

}  // namespace attn
}  // namespace qg
