// The 8-bit paged cache as the kernels see it: E4M3 codes, a power of two for
// kBlock places of a page and head, and their conversions.
#pragma once

#include "kv_batch.cuh"

namespace qg {
namespace kv8 {

constexpr int kBlock = QG_KV8_BLOCK;
constexpr int kBlockShift = 4;
static_assert(1 << kBlockShift == kBlock, "block of a scale");
constexpr int kMinExp = -64, kMaxExp = 63;   // of a scale
constexpr int kBias = 127;                   // of its byte
constexpr float kMost = 448.0f * 9223372036854775808.0f;   // 448 * 2^kMaxExp: a larger value is not kept

struct Cache {
    int num_pages, page_shift, heads, dim;
    long long page_stride, token_stride, head_stride;      // bytes
    long long scale_page, scale_block, scale_head;
};

inline Cache make_cache(const qg_kv8_cache& c)
{
    int sh = 0;
    while ((1 << sh) < c.page_size) sh++;
    return Cache{c.num_pages, sh, c.heads_kv, c.head_dim, c.page_stride, c.token_stride, c.head_stride,
                 c.scale_page_stride, c.scale_block_stride, c.scale_head_stride};
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The least e with amax <= 448 * 2^e, within kMinExp .. kMaxExp (amax <= kMost): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, kMinExp), kMaxExp);
}

// Two values to codes, a in the lower byte; |a|, |b| <= 448, or NaN.
__device__ __forceinline__ uint32_t encode2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// The codes in the lower, or upper, half of w as two fp16 values (exact).
__device__ __forceinline__ uint32_t decode_lo(uint32_t w)
{
    uint32_t r;
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t decode_hi(uint32_t w)
{
    uint32_t r;
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi;}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ float2 half2_floats(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// Four codes, each times 2^down, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float down)
{
    const float2 a = half2_floats(decode_lo(w)), b = half2_floats(decode_hi(w));
    return encode2(a.x * down, a.y * down) | encode2(b.x * down, b.y * down) << 16;
}

// A sequence's new tokens by the blocks of places they fall into.  Work is dealt in units of a block of one sequence, and
// the device finds a unit's sequence without a table of sums: sequence b's units start at cu_q[b] / kBlock + 2 b, which
// leaves it n / kBlock + 2 of them, and n places touch at most (n + 2 kBlock - 2) / kBlock blocks.  With at most one new
// token a sequence, unit b is sequence b.
struct Unit {
    int b, block;       // own places block * kBlock .. + kBlock - 1 (a negative block: places the sequence does not have)
    int t0, s0, s1;     // new tokens at places s0 .. s1 - 1 of the block; the first is row t0
    int page;           // -1: not cached
    bool ok;
};

inline int64_t units_of(const qg_kv_batch& b)
{
    return b.max_q == 1 ? b.sequences : (int64_t)b.tokens / kBlock + 2 * (int64_t)b.sequences;
}

// The unit numbered u, for whole warps; there: it has tokens.  The lengths and offsets of sequences are checked by check_lengths.
__device__ __forceinline__ bool find_unit(const kv::Batch& bt, const Cache& c, int u, Unit& x)
{
    int i = 0, b = u;
    if (bt.max_q != 1) {
        // the last b with cu_q[b] / kBlock + 2 b <= u: a warp looks at 32 places at once (one after another, 8 dependent loads
        // for 256 sequences were 2.6 us of every CTA)
        const int lane = threadIdx.x & 31;
        int lo = 0;
        for (int n = bt.B; n > 1;) {
            const int step = (n + 31) / 32, at = lane * step;
            const bool upto = at < n && (long long)min(max(__ldg(bt.cu_q + lo + at), 0), bt.T) / kBlock + 2LL * (lo + at) <= u;
            const int k = max(__popc(__ballot_sync(0xffffffffu, upto)) - 1, 0);
            lo += k * step;
            n = min(step, n - k * step);
        }
        b = lo;
        const long long first = (long long)min(max(__ldg(bt.cu_q + b), 0), bt.T) / kBlock + 2LL * b;
        if (first > u) return false;
        i = (int)(u - first);
    }
    int t0, t1, len;
    if (!kv::token_range(bt, b, t0, t1) || !kv::own_length(bt, b, len) || t1 <= t0) return false;
    if (i > (t1 - t0) / kBlock + 1) return false;       // rows behind the last sequence
    const int lo = len - (t1 - t0);                     // own place of the first new token
    x.b = b;
    x.block = (lo >> kBlockShift) + i;                  // rounds down below 0 too
    const int p0 = x.block * kBlock;
    if (p0 >= len) return false;
    x.s0 = max(lo - p0, 0);
    x.s1 = min(len - p0, kBlock);
    x.t0 = t0 + p0 + x.s0 - lo;
    x.page = -1;
    if (x.block >= 0) {
        const int e = p0 >> c.page_shift;
        const int page = e < bt.table_ld ? __ldg(bt.table + (long long)b * bt.table_ld + e) : -1;
        if (page >= 0 && page < c.num_pages) x.page = page;
    }
    x.ok = x.page >= 0;
    return true;
}

// Reports lengths and offsets outside their bounds; the grid's threads share the sequences.
__device__ __forceinline__ void check_lengths(const kv::Batch& bt, int* status)
{
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < bt.B; b += gridDim.x * blockDim.x) {
        int t0, t1, len;
        const bool range = kv::token_range(bt, b, t0, t1), length = kv::own_length(bt, b, len);
        if (!range || !length) kv::report(status);
    }
}

}  // namespace kv8
}  // namespace qg
