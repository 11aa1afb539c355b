// What the tile kernels of the 16-bit and the 8-bit cache share: the tensor
// core's operands, tensor memory, and how a CTA walks through its items of work.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attn.cuh"

namespace qg {
namespace attn {
namespace {

constexpr int KB = 128;                      // keys of a block
// The running maximum is only raised when a row's new one is above it by more (in powers of two).
constexpr float kRaise = 8.0f;
constexpr int kTmemCols = 512, kColO = 256;  // S and P of stream s at 128 s, O at 256 + 128 s
template <int X> using Const = std::integral_constant<int, X>;

// kind::f16 instruction descriptor: M = 128, fp32 accumulator; B's head dimension contiguous when `mn`.
template <typename T>
__device__ constexpr uint32_t idesc(int N, bool mn)
{
    const uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
// Upper words of the operands' descriptors (128-byte swizzle); the lower word
// is the address / 16 and the leading offset / 16 << 16, and is advanced by
// 32-bit additions, since all of a product's operands are moved to uniform
// registers for it, and eight products of N = 128 leave 64 clocks for each.
//  K contiguous: rows of 128 bytes, 8-row groups 1024 bytes apart.
//  N contiguous (V): 8 k rows of 64 values are 1024 bytes, the next 8 follow
//  (stride), the next 64 values are a leading offset away.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t leading) { return addr >> 4 | (leading >> 4) << 16; }

// D (+)= A B^T, A from shared or tensor memory.  One lane issues a whole run
// of these inside a branch: electing a lane for each instruction instead
// holds it to one every 77 to 88 clocks (8 steps of K = 16: 655 against 520).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t id, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\t"
                 "mov.b64 b, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
                 "r"(a_low), "r"(b_low), "r"(id), "r"((uint32_t)accumulate), "n"(kDescHigh)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_low, uint32_t id, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(d),
                 "r"(a), "r"(b_low), "r"(id), "r"((uint32_t)accumulate), "n"(kDescHigh)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elect_lane()
{
    uint32_t p;
    asm volatile("{.reg .pred e; elect.sync _|e, 0xffffffff; selp.u32 %0, 1, 0, e;}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
            r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes at once: a whole sector of a thread's own row.
__device__ __forceinline__ void store32(void* p, const uint32_t* r)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z)
{
    float2 r;
    asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; "
        "fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}"
        : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y)
{
    float2 r;
    asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
        : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

// One item: a pair of tiles (or one) of a unit's rows, a key/value head, a part of the keys.
struct Item {
    int head, part;     // part: where partial results go (a piece of the prefix; prompts: a slot)
    int t0, t1;         // first token of the pair, end of the unit's tokens
    bool two;           // the second tile has rows
    int own0;           // own places token t sees: own0 + t - t0
    int own;            // own places any row sees
    int prefix, np;     // prefix tokens, their blocks
    int blk0, blk1;     // this part's blocks
    bool whole;         // all there are
    int b;
};

// Where a CTA is in its work.
struct Cursor {
    int i;      // slot of the deal, or place on the line
    int head;   // next head of the slot (-1 at its start), or of the line
    int pair;   // pair the place on the line lies in
};

// The CTA's next item, or false past the end.
template <int KEYS>
__device__ __forceinline__ bool next_item(const Args& a, const Deal& d, const Layout& lay, Cursor& cur, Item& it)
{
    it.own0 = it.own = 0;
    it.b = 0;
    it.prefix = (KEYS & kPrefix) ? a.bt.prefix_len : 0;
    it.np = (it.prefix + KB - 1) / KB;
    if constexpr (!(KEYS & kOwn)) {
        const int used = kv::used_tokens(a.bt);
        for (; cur.i < d.slots(); cur.i += gridDim.x, cur.head = -1) {
            const bool left = cur.i >= d.pairs * d.groups;   // the single tile
            const int pair = left ? d.pairs : cur.i % d.pairs, G = left ? d.sgroups : d.groups;
            const int g = left ? cur.i - d.pairs * d.groups : cur.i / d.pairs;
            it.t0 = pair * 2 * d.per;
            if (it.t0 >= used) continue;
            const int lo = d.start(g, G), hi = d.start(g + 1, G);
            if (cur.head < 0) cur.head = lo / d.blocks;
            const int base = cur.head * d.blocks;
            if (base >= hi) continue;
            it.t1 = used;
            it.two = used - it.t0 > d.per;
            it.head = cur.head++;
            it.part = g - d.group_of(base, G);
            it.blk0 = max(lo, base) - base;
            it.blk1 = min(hi, base + d.blocks) - base;
            it.whole = false;   // the own tokens are still to be joined
            return true;
        }
        return false;
    } else {
        const Line line = *lay.line;
        const int end = min((int)(blockIdx.x + 1) * line.run, a.c.heads * line.head);
        if (cur.i >= end) return false;
        it.head = cur.head;
        const int at = cur.i - it.head * line.head, lo = cur.pair;
        const Pair p = lay.pair[lo];
        const int blocks = lay.pair[lo + 1].start - p.start, first = it.head * line.head + p.start;   // with the extra ones
        int t0;
        it.b = p.b;
        it.t0 = p.t0;
        kv::token_range(a.bt, p.b, t0, it.t1);
        it.two = it.t1 - it.t0 > lay.per;
        int len;
        kv::own_length(a.bt, p.b, len);   // the layout kernel has reported what is outside its bounds
        it.own0 = len - (it.t1 - it.t0) + 1;
        it.own = max(0, it.own0 + min(2 * lay.per, it.t1 - it.t0) - 1);
        const int u0 = at - p.start, u1 = min(blocks, u0 + end - cur.i);
        it.blk0 = max(0, u0 - lay.extra);
        it.blk1 = max(0, u1 - lay.extra);   // blk0 where the run ends among the extra ones: the piece is written as having seen nothing
        const int from = first / line.run;   // the CTA whose run the item starts in
        it.part = lay.slot(from, (int)blockIdx.x - from);
        it.whole = u0 == 0 && u1 == blocks;
        cur.i += u1 - u0;
        if (++cur.pair == line.pairs) {
            cur.pair = 0;
            cur.head++;
        }
        return true;
    }
}

// Ring positions of an item's loads, in the order K0, K1 V0, K2 V1, ...:
// the order the products want them in.
__device__ __forceinline__ int pos_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int pos_v(int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * j + 1; }

}  // namespace
}  // namespace attn
}  // namespace qg
