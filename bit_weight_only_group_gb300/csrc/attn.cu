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

// How a call is run.
enum Way {
    kAlone,         // row kernel: each sequence over prefix and own tokens
    kRowsShared,    // row kernel: the prefix for all rows and the own tokens in one launch
    kTilesShared,   // tile kernel for the prefix, row kernel for the own tokens beside it
    kPrompts,       // tile kernel: each sequence over prefix and own tokens
};

// How a call is split.  Parts are numbered prefix first.
struct Plan {
    Way way;
    Parts n;        // parts of the row kernel's keys; kTilesShared: most pieces of the prefix
    int parts;      // in all; 1: no joining, results are written at once (kPrompts: 0, its pieces have slots)
    int ctas;       // of the tile kernel
    Deal deal;      // kTilesShared
    int64_t pairs;  // kPrompts: bound of the pairs of tiles of all sequences
};

// Parts of `tiles` tiles for `units` independent units of work: about `ctas`
// CTAs in all, none with fewer than `least` tiles.
void split(int64_t units, int64_t tiles, int64_t ctas, int least, int* parts, int* per)
{
    const int64_t want = std::max<int64_t>(1, ceil_div(ctas, std::max<int64_t>(1, units)));
    const int64_t n = std::min(want, std::max<int64_t>(1, tiles / least));
    *per = (int)std::max<int64_t>(1, ceil_div(tiles, n));
    *parts = (int)std::max<int64_t>(1, ceil_div(tiles, *per));
}

// The shared prefix dealt to `ctas` CTAs, none with less than two blocks.
Deal make_deal(const qg_kv_cache& c, const qg_kv_batch& b, int64_t group, int ctas)
{
    Deal d{};
    d.per = tile_tokens(group);
    d.heads = c.heads_kv;
    d.blocks = (int)ceil_div(b.prefix_len, kBlock);
    const int64_t line = (int64_t)d.heads * d.blocks, tiles = ceil_div(b.tokens, d.per);
    const int64_t most = std::max<int64_t>(1, std::min(line / 2, ((int64_t)1 << 31) / line - 1));
    d.pairs = (int)(tiles / 2);
    d.single = (int)(tiles % 2);
    // CTAs in proportion to the work: a pair of tiles 2, a single one 1
    if (d.pairs) d.groups = (int)std::min<int64_t>(most, std::max<int64_t>(1, 2 * (int64_t)ctas / tiles));
    if (d.single) d.sgroups = (int)std::min<int64_t>(most, std::max<int64_t>(1, ctas - (int64_t)d.pairs * d.groups));
    return d;
}

// Microseconds the row kernel takes on the whole card for the own tokens,
// which fill half of max_kv, say: 6.4 TB/s, or, with more than 16 rows a
// sequence and head, 0.7 an SM for each 32 rows and 64 keys.
double own_time(const qg_kv_cache& c, const qg_kv_batch& b, int64_t group)
{
    const double pairs = 0.5 * b.sequences * c.heads_kv, rows = (double)group * b.max_q;
    const double bytes = pairs * b.max_kv * c.head_dim * 4 / 6.4e6;
    const double products = rows > 16 ? pairs * ceil_div((int64_t)rows, 32) * ceil_div(b.max_kv, kTile) * 0.7 / num_sms() : 0.0;
    return 5.0 + std::max(bytes, products);
}

// Microseconds the tile kernel takes on an SM for a block and so many tiles:
// 1.35 for a pair, 1.2 for a single tile (bound by its loads), two thirds of
// that with 64-wide heads.
double block_time(const qg_kv_cache& c, int64_t tiles)
{
    return (c.head_dim == 128 ? 1.0 : 0.67) * ((double)(tiles / 2) * 1.35 + (double)(tiles % 2) * 1.2);
}

// CTAs (one an SM) for the shared prefix, so that the own tokens' kernel, which
// runs beside on the other SMs and takes over the rest when they end, ends
// with them.  A CTA of the tile kernel takes about 10 us before and after its
// blocks, and is slowed by up to 0.7 where the other kernel has the memory;
// the row kernel takes 0.006 us a CTA.  Measured over 32 to 152 CTAs: 256
// sequences over 8192 + 1024 keys best at 64 (134 us, 158 on all SMs), 64 over
// 32768 + 2048 at 96 to 112 (103, 120), 128 over 131072 + 2048 at 136 (429,
// 446), 32 over 2011 + 700 with a key/value head per query head at 32 (48, 56).
//
// Lengths far below max_kv leave the SMs kept for the own tokens idle early, so
// the prefix gets no fewer CTAs than make it take kSlowest times as long as all
// of them would.
constexpr double kSlowest = 2.25;
int choose_ctas(const qg_kv_cache& c, const qg_kv_batch& b, int64_t group, int64_t own_ctas)
{
    const int all = num_sms();
    const double sms = all;
    const double own = own_time(c, b, group) + 0.006 * own_ctas;
    int best = all;
    double least = 1e30, on_all = 0.0;
    for (int x = all; x >= 8; x -= 4) {
        const Deal d = make_deal(c, b, group, x);
        const double line = (double)d.heads * d.blocks, rounds = (double)ceil_div(d.slots(), x);
        const double each = rounds * std::max(d.pairs ? block_time(c, 2) * line / d.groups : 0.0,
                                              d.single ? block_time(c, 1) * line / d.sgroups : 0.0);
        if (x == all) on_all = 10.0 + each;
        if (10.0 + each > kSlowest * on_all) continue;
        const double busy = std::min(x, d.slots());
        const double tile_end = (10.0 + each) * (1.0 + 0.7 * (sms - busy) / sms);
        const double all_end = own + (10.0 + each) * busy / sms;
        const double end = std::max(tile_end, all_end);
        if (end < least) {
            least = end;
            best = x;
        }
    }
    return best;
}

// The line of prompts is counted in 32 bits.
bool line_fits(const qg_kv_cache& c, const qg_kv_batch& b, int64_t per2)
{
    const int64_t pairs = b.tokens / per2 + b.sequences;
    return pairs * (ceil_div(b.prefix_len, kBlock) + ceil_div(b.max_kv, kBlock) + 1) < ((int64_t)1 << 30) / c.heads_kv;
}

Plan make_plan(const qg_kv_cache& c, const qg_kv_batch& b, int heads_q)
{
    Plan p{};
    const int64_t group = heads_q / c.heads_kv, sms = num_sms();
    const int64_t per = std::max(1, tile_tokens(group)), rows = group * b.tokens;
    const int64_t np = ceil_div(b.prefix_len, kBlock), no = ceil_div(b.max_kv, kBlock);
    const int64_t prefix_tiles = ceil_div(b.prefix_len, kTile), own_tiles = ceil_div(b.max_kv, kTile);
    const int64_t own_units = (int64_t)b.sequences * c.heads_kv * ceil_div(group * b.max_q, 64);
    const bool tiles = group <= 128;   // a tile holds whole tokens
    const bool share = b.sequences > 1 && b.prefix_len >= 256;
    p.way = share ? kTilesShared : kAlone;
    if (share) {
        // little work on the prefix, in blocks of 64 rows and 64 keys over the heads, is done sooner by the row kernel,
        // which starts sooner and needs one launch less (512 blocks: 128 rows over 2048 keys of 8 heads 19.3 us, 20.8 by
        // tiles; 1024 blocks: 64 rows over 8192 keys 28.2, 24.5), and longer where it is bound by the keys (16 rows over
        // 8192 keys 14.6, 23.7)
        const int64_t work = c.heads_kv * ceil_div(rows, 64) * prefix_tiles;
        if (!tiles || work <= (rows <= 16 ? 4096 : 600)) p.way = kRowsShared;
    }
    if (tiles && group * b.max_q > 64 && line_fits(c, b, 2 * per)) {
        // rows enough for tiles within a sequence: prefix and own tokens in one pass, unless packing the rows of all
        // sequences into tiles for the prefix saves more than the row kernel costs for the own tokens
        const int64_t each = std::min<int64_t>(ceil_div(b.max_q, per), ceil_div(b.tokens, per * std::max(1, b.sequences)));
        const double apart = b.sequences * c.heads_kv * block_time(c, each) * (np + 0.5 * no) / sms;
        const double packed = c.heads_kv * block_time(c, ceil_div(b.tokens, per)) * np / sms + own_time(c, b, group);
        if (!share || apart <= packed) p.way = kPrompts;
        else p.way = kTilesShared;
    }
    switch (p.way) {
        case kAlone:
            split(own_units, prefix_tiles + own_tiles, 3 * sms, kLeastTiles, &p.n.own_parts, &p.n.own_tiles);
            break;
        case kRowsShared: {
            const int64_t units = c.heads_kv * ceil_div(rows, 64);
            split(units, prefix_tiles, sms, 2, &p.n.prefix_parts, &p.n.prefix_tiles);
            split(own_units, own_tiles, 3 * sms, kLeastTiles, &p.n.own_parts, &p.n.own_tiles);
            break;
        }
        case kTilesShared:
            split(own_units, own_tiles, 4 * sms, kLeastTiles, &p.n.own_parts, &p.n.own_tiles);
            p.ctas = choose_ctas(c, b, group, own_units * p.n.own_parts);
            p.deal = make_deal(c, b, group, p.ctas);
            p.n.prefix_parts = p.deal.most_pieces();
            break;
        case kPrompts: {
            p.pairs = b.tokens / (2 * per) + b.sequences;
            p.ctas = (int)std::min<int64_t>(sms, ceil_div(c.heads_kv * p.pairs * std::max<int64_t>(1, np + no), kMinRun));
            break;
        }
    }
    p.parts = p.n.prefix_parts + p.n.own_parts;
    return p;
}

// The workspace: o of the parts, (m, l) of the parts, the layout of prompts.
struct Places {
    size_t ml, line, first, pair, cut, bytes;
};
Places places(const Plan& p, const qg_kv_batch& b, int heads_q, int dim)
{
    Places w{};
    size_t rows = p.parts * (size_t)b.tokens * heads_q;
    if (p.way == kPrompts) {
        // The slots of the CTAs' pieces: 41 MB with heads of 128 on 152 SMs, however long the prompts are.  Short
        // prompts are asked for two parts of each row, up to 2^18 rows (139 MB), whether the slots fill that or not: a
        // size that callers may have fixed, and that grows with the prompt no further.
        rows = std::max((size_t)2 * p.ctas * kSlotRows, std::min<size_t>(2 * (size_t)b.tokens * heads_q, (size_t)1 << 18));
    } else if (p.parts <= 1) {
        return w;
    }
    w.ml = align_up(rows * dim * 4, 256);
    w.line = w.ml + align_up(rows * sizeof(float2), 256);
    w.bytes = w.line;
    if (p.way == kPrompts) {
        w.first = w.line + align_up(sizeof(Line), 256);
        w.pair = w.first + align_up((size_t)(b.sequences + 1) * 4, 256);
        w.cut = w.pair + align_up((size_t)(p.pairs + 1) * sizeof(Pair), 256);
        w.bytes = w.cut + align_up((size_t)p.ctas * 4, 256);
    }
    return w;
}

// out[r] = sum_p w_p o_p / sum_p w_p l_p with w_p = 2^(m_p - max m), in the
// order of the parts: dim / 8 lanes a row, 8 of its values a lane.  slot(p) is
// the place of part p's row.  Bound by latency
// (the parts were just written and are in L2): the (m, l) and the values of
// the first AT_ONCE parts are loaded at once, before anything that decides
// whether they are wanted.  Few rows take eight parts at once; many take two,
// in 48 registers, so that more rows run in a round.
template <int D, int AT_ONCE, typename Slot>
__device__ __forceinline__ void join_row(const Args& a, int t, int hq, int n, const int* used, Slot slot)
{
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x % LANES;
    const uint32_t mask = (LANES == 32 ? 0xffffffffu : (1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
    const long long row = (long long)t * a.heads_q + hq;
    auto load_ml = [&](int p) { return p < n ? __ldcg(a.part_ml + slot(p)) : make_float2(-INFINITY, 0.0f); };
    float4 v[AT_ONCE][2];
    auto load_o = [&](int p0) {   // where a part saw nothing its values are unset, and are not used
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++)
            if (p0 + i < n) {
                const float4* src = reinterpret_cast<const float4*>(a.part_o + slot(p0 + i) * D) + 2 * lane;
                v[i][0] = __ldcg(src);
                v[i][1] = __ldcg(src + 1);
            }
    };
    float2 ml = load_ml(lane);
    load_o(0);
    const bool mine = t < (used ? min(max(__ldg(used), 0), a.bt.T) : a.bt.T);
    float m = ml.y != 0.0f ? ml.x : -INFINITY, l = 0.0f;
    for (int p = LANES + lane; p < n; p += LANES) {
        const float2 w = load_ml(p);
        if (w.y != 0.0f) m = fmaxf(m, w.x);
    }
#pragma unroll
    for (int i = LANES / 2; i > 0; i /= 2) m = fmaxf(m, __shfl_xor_sync(mask, m, i, LANES));
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; e++) o[e] = 0.0f;
    float w = ml.y != 0.0f ? exp2_approx(ml.x - m) : 0.0f;
    for (int p0 = 0; p0 < n; p0 += AT_ONCE) {
        if (p0 && p0 % LANES == 0) {
            ml = load_ml(p0 + lane);
            w = ml.y != 0.0f ? exp2_approx(ml.x - m) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            const float wp = __shfl_sync(mask, w, (p0 + i) % LANES, LANES);
            const float lp = __shfl_sync(mask, ml.y, (p0 + i) % LANES, LANES);
            if (p0 + i < n && lp != 0.0f) {
                l = fmaf(wp, lp, l);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    o[4 * h] = fmaf(wp, v[i][h].x, o[4 * h]);
                    o[4 * h + 1] = fmaf(wp, v[i][h].y, o[4 * h + 1]);
                    o[4 * h + 2] = fmaf(wp, v[i][h].z, o[4 * h + 2]);
                    o[4 * h + 3] = fmaf(wp, v[i][h].w, o[4 * h + 3]);
                }
            }
        }
        load_o(p0 + AT_ONCE);
    }
    if (!mine) return;
    const float inv = inverse(l);
    uint32_t bits[8];
#pragma unroll
    for (int e = 0; e < 8; e++) bits[e] = __float_as_uint(o[e] * inv);
    store_out8(a, t * a.ldo + (long long)hq * D + 8 * lane, bits);
    if (lane == 0) store_lse(a, row, m, l);
}
template <int D> constexpr int kJoinRows = 256 / (D / 8);   // rows of a joining CTA

// All rows: the prefix's pieces first, then the other parts.
template <int D, int AT_ONCE>
__global__ void __launch_bounds__(256, AT_ONCE == 2 ? 5 : 2) k_attn_join(const __grid_constant__ Args a, const __grid_constant__ Deal d,
                                                      int part0, int parts)
{
    kv::pdl_wait();
    kv::pdl_release();
    const uint32_t row = blockIdx.x * kJoinRows<D> + threadIdx.x / (D / 8);
    if (row >= a.rows) return;
    const int t = (int)(row / (uint32_t)a.heads_q), hq = (int)row - t * a.heads_q;
    int pieces = 0;
    if (d.blocks) pieces = d.pieces(hq / a.group, t < d.pairs * 2 * d.per ? d.groups : d.sgroups);
    join_row<D, AT_ONCE>(a, t, hq, pieces + parts, a.bt.cu_q ? a.bt.cu_q + a.bt.B : nullptr,
                         [&](int p) { return (long long)(p < pieces ? p : part0 + p - pieces) * a.rows + row; });
}

// The rows of items that the end of a CTA's run cut: kCutCtas CTAs for the 256
// rows at each run's end, which leave the item to its first cut.  (Four rounds
// of rows a CTA: with one, 151 cuts take three waves of CTAs.)
constexpr int kCutCtas = 4;
template <int D>
__global__ void __launch_bounds__(256, 5) k_attn_join_line(const __grid_constant__ Args a, const __grid_constant__ Layout lay)
{
    kv::pdl_wait();
    kv::pdl_release();
    const Line line = *lay.line;
    const int c = blockIdx.x / kCutCtas + 1, lo = lay.cut[c];
    if ((long long)c * line.run >= (long long)a.c.heads * line.head) return;
    const int head = c * line.run / line.head, at = c * line.run - head * line.head;
    const Pair p = lay.pair[lo];
    const int first = head * line.head + p.start, last = head * line.head + lay.pair[lo + 1].start - 1;
    if (p.start == at || first / line.run != c - 1) return;
    int t0, t1;
    kv::token_range(a.bt, p.b, t0, t1);
    const int n = last / line.run - (c - 1) + 1, tile_rows = lay.per * a.group;
    for (int r = blockIdx.x % kCutCtas * (256 / kCutCtas) + threadIdx.x / (D / 8); r < (blockIdx.x % kCutCtas + 1) * (256 / kCutCtas);
         r += kJoinRows<D>) {
        const int t = p.t0 + r / a.group;
        if (r >= 2 * tile_rows || t >= t1) return;
        const int at = r < tile_rows ? r : 128 + r - tile_rows;
        join_row<D, 2>(a, t, head * a.group + r % a.group, n, nullptr,
                       [&](int p) { return (long long)lay.slot(c - 1, p) * kSlotRows + at; });
    }
}

}  // namespace

cudaError_t launch_join(const Args& a, const Deal& d, int part0, int parts, cudaStream_t s)
{
    const int each = a.c.dim == 128 ? kJoinRows<128> : kJoinRows<64>;
    const dim3 grid((unsigned)ceil_div(a.rows, each));
    const bool few = grid.x <= 2u * num_sms();   // one round of the wide form: 1024 rows of 13 parts 6.2 us, 8.0 in the narrow
    if (a.c.dim == 128)
        return few ? kv::launch_dependent(k_attn_join<128, 8>, grid, 256, 0, s, a, d, part0, parts)
                   : kv::launch_dependent(k_attn_join<128, 2>, grid, 256, 0, s, a, d, part0, parts);
    return few ? kv::launch_dependent(k_attn_join<64, 8>, grid, 256, 0, s, a, d, part0, parts)
               : kv::launch_dependent(k_attn_join<64, 2>, grid, 256, 0, s, a, d, part0, parts);
}

cudaError_t launch_join_line(const Args& a, const Layout& lay, cudaStream_t s)
{
    const dim3 grid((unsigned)(kCutCtas * (lay.ctas - 1)));
    if (!grid.x) return cudaSuccess;
    return a.c.dim == 128 ? kv::launch_dependent(k_attn_join_line<128>, grid, 256, 0, s, a, lay)
                          : kv::launch_dependent(k_attn_join_line<64>, grid, 256, 0, s, a, lay);
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
    const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
    const CUresult r = fn(map, dtype == QG_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(QG_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return QG_OK;
}
}  // namespace

qg_status encode_pages(CUtensorMap* map, const qg_kv_cache& c, const void* base, int box_rows, bool whole)
{
    // the stride of a dimension of one entry is never used: any valid one
    const cuuint64_t any = 16, token = (cuuint64_t)c.token_stride * 2;
    const cuuint64_t head = c.heads_kv > 1 ? (cuuint64_t)c.head_stride * 2 : any;
    const cuuint64_t page = c.num_pages > 1 ? (cuuint64_t)c.page_stride * 2 : any;
    const cuuint64_t places = c.page_size, heads = c.heads_kv, pages = c.num_pages, halves = c.head_dim / 64;
    if (whole) {
        const cuuint64_t dims[5] = {64, places, halves, heads, pages}, strides[4] = {token, 128, head, page};
        const cuuint32_t box[5] = {64u, (cuuint32_t)box_rows, (cuuint32_t)halves, 1u, 1u};
        return encode(map, c.dtype, 5, base, dims, strides, box);
    }
    const cuuint64_t dims[4] = {64 * halves, places, heads, pages}, strides[3] = {token, head, page};
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
    return attn::places(attn::make_plan(cache, batch, heads_q), batch, heads_q, cache.head_dim).bytes;
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
    const attn::Places w = attn::places(p, batch, heads_q, cache.head_dim);
    char* base = static_cast<char*>(ws);
    a.part_o = w.bytes ? reinterpret_cast<float*>(base) : nullptr;
    a.part_ml = w.bytes ? reinterpret_cast<float2*>(base + w.ml) : nullptr;
    a.status = device_status_ptr();
    qg_status st = QG_OK;
    CUtensorMap qmap, kmap, vmap;
    cudaError_t e = cudaSuccess;
    if (p.way == attn::kTilesShared || p.way == attn::kPrompts) {
        a.box_rows = std::min(cache.page_size, attn::kBlock / 2);
        st = attn::encode_rows(&qmap, cache.dtype, q, cache.head_dim, heads_q, ldq, batch.tokens, a.group);
        if (st == QG_OK) st = attn::encode_pages(&kmap, cache, cache.k, a.box_rows, false);
        if (st == QG_OK) st = attn::encode_pages(&vmap, cache, cache.v, a.box_rows, false);
        if (st != QG_OK) return st;
        if (p.way == attn::kPrompts) {
            const attn::Layout lay{reinterpret_cast<attn::Line*>(base + w.line), reinterpret_cast<int*>(base + w.first),
                                   reinterpret_cast<attn::Pair*>(base + w.pair), reinterpret_cast<int*>(base + w.cut),
                                   attn::tile_tokens(a.group), p.ctas, (int)p.pairs};
            e = attn::launch_tiles(a, cache.dtype, qmap, kmap, vmap, lay, s);
            if (e == cudaSuccess) e = attn::launch_join_line(a, lay, s);
        } else {
            e = attn::launch_tiles_shared(a, cache.dtype, qmap, kmap, vmap, p.deal, p.ctas, s);
        }
    }
    if (p.way != attn::kPrompts && e == cudaSuccess) {
        a.box_rows = std::min(cache.page_size, attn::kTile);
        st = attn::encode_pages(&kmap, cache, cache.k, a.box_rows, true);
        if (st == QG_OK) st = attn::encode_pages(&vmap, cache, cache.v, a.box_rows, true);
        if (st != QG_OK) return st;
        if (p.way == attn::kRowsShared) e = attn::launch_rows_shared(a, cache.dtype, kmap, vmap, p.n, s);
        else if (p.way == attn::kTilesShared) e = attn::launch_rows(a, cache.dtype, kmap, vmap, attn::kOwn, p.n, true, s);
        else e = attn::launch_rows(a, cache.dtype, kmap, vmap, attn::kPrefix | attn::kOwn, p.n, false, s);
        // the deal's pieces come first; parts of the row kernel alone follow one another from 0 on
        if (e == cudaSuccess && p.parts > 1)
            e = p.way == attn::kTilesShared ? attn::launch_join(a, p.deal, p.n.prefix_parts, p.n.own_parts, s)
                                            : attn::launch_join(a, p.deal, 0, p.parts, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "qattn_forward launch");
    return QG_OK;
}

}  // namespace qg
