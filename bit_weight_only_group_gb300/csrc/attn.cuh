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

#include "kv8.cuh"
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
    // partial results: o of part p, row r at part_o + (p * rows + r) * dim, (m, l) at part_ml + p * rows + r;
    // those of prompts in slots of 256 rows (Layout)
    float* part_o;
    float2* part_ml;
    long long rows;              // T * heads_q
    int box_rows;                // key rows of one TMA box of the kernel launched
    int* status;
};

// Attention over the 8-bit cache: a.c's strides count bytes, a.q is of type q_type.
//
// The products are in fp16, which holds the codes exactly.  A row of q is scaled
// by a power of two to below 2^15 (its lower bits, down to 2^-39 of the row's
// largest value, stay), and the K scale goes on the logits in fp32.  The V scale
// 2^ev goes into the exponent: P' = 2^(s + ev - m) with m the maximum of s + ev,
// so that P' codes sum to 2^-m sum 2^s v, and l = sum 2^-ev P' (fp32) is 2^-m sum
// 2^s: parts as above, but that m is not the largest s.  P' is rounded to fp16.
struct Args8 {
    Args a;
    const uint8_t *k_codes, *v_codes;
    const uint8_t *k_scale, *v_scale;
    long long scale_page, scale_block, scale_head;
    int q_type;
};
// Scales are looked up in two steps, the page of 16 keys and the byte there, each some rounds ahead of its use.  Both are
// loaded whether there is something to look up or not (from a place that is there), and first looked at where they are
// used: a choice or a comparison after the load would wait for it.
struct Entry {
    int page;      // as the table has it
    bool there;    // there are keys to look up
};
// Entry e of a table (lengths are cut to bounds that the host has checked against the tables).
__device__ __forceinline__ Entry table_entry(const Args& a, const int* table, int e, bool there)
{
    return Entry{__ldg(there ? table + e : a.bt.kv_len), there};
}
// The page an entry names; num_pages where it is not to be followed, -1 where there was none to look up.
__device__ __forceinline__ int checked_page(const Args& a, const Entry& e)
{
    if (!e.there) return -1;
    if (e.page >= 0 && e.page < a.c.num_pages) return e.page;
    kv::report(a.status);
    return a.c.num_pages;
}
// Byte of the scale of a K or V block in a checked page; any block's where there is none (its keys count for nothing).
__device__ __forceinline__ int scale_byte(const Args8& p, bool v, int page, int block, int head)
{
    const long long at = (long long)page * p.scale_page + (long long)block * p.scale_block + (long long)head * p.scale_head;
    return (int)__ldg((v ? p.v_scale : p.k_scale) + (page >= 0 && page < p.a.c.num_pages ? at : 0));
}
// Its exponent (a byte outside 1 .. 254 is none the appending kernel wrote).
__device__ __forceinline__ int scale_exp(int byte) { return min(max(byte, 1), 254) - kv8::kBias; }
// The power of two 2^x that brings a row with the largest magnitude amax to 2^14 .. 2^15 is 2^(14 - x).
__device__ __forceinline__ int row_exp(float amax) { return max((int)(__float_as_uint(amax) >> 23) - 127, -100); }

constexpr float kLn2 = 0.69314718055994530942f;

// Values of a finished row.
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
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
            a.out_type == QG_T_BF16 ? make_uint2(kv::pack2<__nv_bfloat16>(v.x, v.y), kv::pack2<__nv_bfloat16>(v.z, v.w))
                                    : make_uint2(kv::pack2<__half>(v.x, v.y), kv::pack2<__half>(v.z, v.w));
}
// Eight fp32 values (as bits).
__device__ __forceinline__ void store_out8(const Args& a, long long at, const uint32_t* v)
{
    const float* f = reinterpret_cast<const float*>(v);
    if (a.out_type == QG_T_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint4 w;
        if (a.out_type == QG_T_BF16)
            w = make_uint4(kv::pack2<__nv_bfloat16>(f[0], f[1]), kv::pack2<__nv_bfloat16>(f[2], f[3]),
                           kv::pack2<__nv_bfloat16>(f[4], f[5]), kv::pack2<__nv_bfloat16>(f[6], f[7]));
        else
            w = make_uint4(kv::pack2<__half>(f[0], f[1]), kv::pack2<__half>(f[2], f[3]), kv::pack2<__half>(f[4], f[5]),
                           kv::pack2<__half>(f[6], f[7]));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) = w;
    }
}
// A sum l of 0 says that nothing was seen.  A NaN among the logits makes l a
// NaN, which is not 0: such a row, or part of one, is kept and stays a NaN.
__device__ __forceinline__ float inverse(float l) { return l != 0.0f ? 1.0f / l : 0.0f; }
__device__ __forceinline__ void store_lse(const Args& a, long long row, float m, float l)
{
    if (a.lse) a.lse[row] = l != 0.0f ? kLn2 * (m + log2f(l)) : -INFINITY;
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

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
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
// Maps of K or V pages.  whole: dimensions (64 values, place, half of the
// head, head, page), boxes of box_rows places of a whole head; else (dim,
// place, head, page), boxes of 64 values x box_rows places.
qg_status encode_pages(CUtensorMap* map, const qg_kv_cache& c, const void* base, int box_rows, bool whole);
// Map of 8-bit K or V pages: dimensions (dim, place, head, page), boxes of box_rows places of a whole head.
qg_status encode_pages8(CUtensorMap* map, const qg_kv8_cache& c, const void* base, int box_rows);
// Map of the query rows: dimensions (dim, head, token), boxes of 64 values x a group x a tile's tokens.
qg_status encode_rows(CUtensorMap* map, int dtype, const void* q, int dim, int heads_q, int64_t ldq, int64_t tokens,
                      int group);

// How the tile kernel's work on a shared prefix is dealt: a pair of tiles
// (256 rows) is worked on by `groups` CTAs, each taking an equal run of the
// blocks of all heads laid end to end, so a head's blocks fall into pieces, one
// part each.  CTAs of different pairs in the same group run over the same
// blocks at the same time and share their loads in L2.  A last, single tile
// (half the work) has groups of its own.
struct Deal {
    int per;                  // tokens of a tile
    int pairs, groups;        // full pairs of tiles
    int single, sgroups;      // 1: a tile is left over, and its groups
    int blocks;               // blocks of a head
    int heads;
    // (every product below fits 32 bits: launches keep line * CTAs below 2^31)
    __host__ __device__ uint32_t line() const { return (uint32_t)heads * blocks; }
    __host__ __device__ int slots() const { return pairs * groups + (single ? sgroups : 0); }
    // first block of group g of G, and the group a block belongs to
    __host__ __device__ int start(uint32_t g, uint32_t G) const { return (int)(g * line() / G); }
    __host__ __device__ int group_of(uint32_t block, uint32_t G) const { return (int)(((block + 1) * G - 1) / line()); }
    // pieces of head h, and a bound for any head
    __host__ __device__ int pieces(int h, int G) const
    {
        return group_of((h + 1) * blocks - 1, G) - group_of(h * blocks, G) + 1;
    }
    __host__ __device__ int most_pieces() const
    {
        const int G = single && sgroups > groups ? sgroups : groups;
        const int n = (G + heads - 1) / heads + 1;
        return n < blocks ? n : blocks;
    }
};

// How the tile kernel's work on prompts is dealt.  The pairs of tiles of all
// sequences, each with the blocks its last token sees, are laid end to end for
// a head, the heads after one another, and each CTA takes an equal run of
// that line.  An item (a pair, a head) inside one run is written at once; one
// that runs cross falls into pieces, joined afterwards.  A CTA has at most two
// pieces, one of an item that starts before its run and one of an item that
// starts in it and ends after it, so two slots of a pair's 256 rows a CTA hold
// them all.  The lengths are on the device, so a small kernel lays the line out.
struct Line {
    int run;                  // blocks of a CTA
    int head;                 // blocks of a head
    int pairs;
};
struct Pair {
    int start;                // blocks of a head before it
    int t0;                   // its first token
    int b;                    // its sequence
};
struct Layout {
    Line* line;
    int* first;               // [B + 1] pairs before each sequence
    Pair* pair;               // [pairs + 1], the last one's start the end of the line
    int* cut;                 // [ctas] pair in which the run of each CTA starts
    int per;                  // tokens of a tile
    int ctas;
    int max_pairs;            // entries of `pair` but one
    int extra;                // blocks that an item's start and end count for, before its first
    // slot of piece p of an item that starts in the run of CTA c
    __host__ __device__ int slot(int c, int p) const { return p == 0 ? 2 * c + 1 : 2 * (c + p); }
};
constexpr int kSlotRows = 256;   // the first tile's 128, the second's
constexpr int kMinRun = 2;       // blocks: a CTA's start and end cost several
constexpr int kMostPieces = 32;  // of an item: joining takes them two at a time, one after another

// The kernels' launches.  A keys flag says what a row sees: the shared
// prefix, its own sequence's tokens, or both in that order.
enum Keys { kPrefix = 1, kOwn = 2 };
// Parts of the keys and most tiles (64 keys) of one, for the row kernel; own: of
// the own tokens, or of prefix and own tokens together.  Parts of the prefix
// come first.  The tiles there are, which only the device knows, are dealt
// evenly to the parts, at least kLeastTiles to one; beside the tile kernel at
// least kLeastBeside, since there the SMs' time counts, and a CTA's start and
// end take some of it (64 sequences over 32768 + 32 to 2048 own tokens 100 us,
// 105 with kLeastTiles; 48 of 5 drafted tokens 38, 40.5).
struct Parts {
    int prefix_parts, prefix_tiles, own_parts, own_tiles;
};
constexpr int kLeastTiles = 4, kLeastBeside = 16;
// beside: launched right after the tile kernel of the same call, whose results it does not use, to run at its side.
cudaError_t launch_rows(const Args& a, int dtype, const CUtensorMap& kmap, const CUtensorMap& vmap, int keys,
                        const Parts& p, bool beside, cudaStream_t s);
// The shared prefix for all rows and the own tokens in one launch.
cudaError_t launch_rows_shared(const Args& a, int dtype, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& p,
                               cudaStream_t s);
// The same two over the 8-bit cache.
cudaError_t launch_rows8(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int keys, const Parts& n,
                         bool beside, cudaStream_t s);
cudaError_t launch_rows8_shared(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& n,
                                cudaStream_t s);
// Tokens of a tile of the tile kernel (its rows: that times the group, at most 128).
inline int tile_tokens(int64_t group) { return (int)(128 / group); }
// The shared prefix for all tokens, dealt to at most `ctas` CTAs, parts 0 .. most_pieces() - 1.
cudaError_t launch_tiles_shared(const Args& a, int dtype, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, const Deal& d, int ctas, cudaStream_t s);
// Each sequence's tokens over prefix and own tokens: lays the line out and works through it.
cudaError_t launch_tiles(const Args& a, int dtype, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, const Layout& lay, cudaStream_t s);
// Lays the line of prompts out.
cudaError_t launch_layout(const Args& a, const Layout& lay, cudaStream_t s);
// The tile kernel over the 8-bit cache (the line of prompts laid out before).
cudaError_t launch_tiles8_shared(const Args8& p, const Deal& d, int ctas, cudaStream_t s);
cudaError_t launch_tiles8(const Args8& p, const Layout& lay, cudaStream_t s);
// Joins, for each row, the pieces of `d` (none when d.blocks = 0) and `parts` parts from part0 on.
cudaError_t launch_join(const Args& a, const Deal& d, int part0, int parts, cudaStream_t s);
// Joins the items of a line that fell into pieces.
cudaError_t launch_join_line(const Args& a, const Layout& lay, cudaStream_t s);

}  // namespace attn
}  // namespace qg
