// What the row kernels of the 16-bit and the 8-bit cache share: what a CTA works
// on, how a launch is split, and the warp-level matrix instructions.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attn.cuh"

namespace qg {
namespace attn {
namespace {

constexpr int KT = 64;                       // keys of a stage of the 16-bit kernel
constexpr int kWarps = 4;                    // consumer warps; warp 4 issues the loads
constexpr int kThreads = (kWarps + 1) * 32;

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
static_assert(kWarps * 32 == 128, "consumer_sync counts 128 threads");

// What one CTA works on.
struct Item {
    int t0;             // the unit's first token; its row i is query head i % group of token t0 + i / group
    int row0, rows;     // this CTA's rows of it
    int b;              // sequence (own keys only)
    int own0;           // own places token t sees: own0 + t - t0 (own keys only)
    int own;            // own places any row sees
    int prefix, np;     // prefix tokens and their tiles (0 without prefix keys)
    int tile0, tile1;   // this part's tiles
};

template <int KEYS, int TILE>   // TILE: keys of a tile
__device__ __forceinline__ Item find_item(const Args& a, int unit, int row_block, int part, int parts, int least_tiles,
                                          int rows_cap, bool tell)
{
    Item it;
    it.b = unit;
    int t0, t1;
    bool ok = true;
    if (KEYS & kOwn) {
        ok = kv::token_range(a.bt, unit, t0, t1);
    } else {
        t0 = 0;
        t1 = kv::used_tokens(a.bt);
    }
    it.t0 = t0;
    it.row0 = row_block * rows_cap;
    it.rows = max(0, min(rows_cap, (t1 - t0) * a.group - it.row0));
    it.own = it.own0 = 0;
    if ((KEYS & kOwn) && it.rows > 0) {
        int len;
        ok = kv::own_length(a.bt, unit, len) && ok;
        it.own0 = len - (t1 - t0) + 1;
        it.own = max(0, it.own0 + (it.row0 + it.rows - 1) / a.group);
    }
    if (!ok && tell) kv::report(a.status);
    it.prefix = (KEYS & kPrefix) ? a.bt.prefix_len : 0;
    it.np = (it.prefix + TILE - 1) / TILE;
    const int tiles = it.rows > 0 ? it.np + (it.own + TILE - 1) / TILE : 0;
    const int per = max(least_tiles, (tiles + parts - 1) / parts);
    it.tile0 = min(part * per, tiles);
    it.tile1 = min(it.tile0 + per, tiles);
    return it;
}

// The CTA numbered x of a launch's (unit, row block, part, head) CTAs.
struct Split {
    int part0, parts, least_tiles, row_blocks;
};

// Row blocks of 16 rows that a CTA takes for so many rows a unit.
int row_warps(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

struct Launch {
    Split sp;
    int64_t ctas;
};
// most_tiles: of 64 keys, of a part; tile: keys of the kernel's tiles.
Launch plan(const Args& a, int keys, int rw, int part0, int parts, int most_tiles, bool beside = false, int tile = KT)
{
    const int64_t units = (keys & kOwn) ? a.bt.B : 1;
    const int64_t blocks = ceil_div((int64_t)a.group * ((keys & kOwn) ? a.bt.max_q : a.bt.T), 16 * rw);
    const int least = (int)ceil_div(std::min(beside ? kLeastBeside : kLeastTiles, most_tiles), tile / 64);
    return Launch{Split{part0, parts, least, (int)blocks}, units * blocks * parts * a.c.heads};
}

}  // namespace
}  // namespace attn
}  // namespace qg
