// Attention for many query rows per key/value head on the 5th-generation
// tensor cores: the prefix shared by a batch (all its tokens' rows against one
// run of keys), and prompts of many tokens a sequence.
//
// A tile is up to 128 rows: 128 / group tokens times the query heads of one
// key/value head.  Keys come in blocks of 128.  For a tile and a block
//     S = Q K^T     tcgen05, Q and K from shared memory, S in tensor memory
//     P = 2^(S scale_log2 - m)   one thread a row: S read from tensor memory,
//                   P written back over it in the cache's type (16-bit operands
//                   of the next product; the sum l is of P before that rounding,
//                   whose error attn_rows.cu gives)
//     O += P V      tcgen05, P from tensor memory, V from shared memory
//                   (its head dimension contiguous), O in tensor memory
// The tensor core waits for the softmax of a block and the softmax for its S,
// so a CTA runs two such chains ("streams") side by side, 256 columns of
// tensor memory each (S and P 128, O 128): while one is in its softmax the
// tensor core works for the other.  With two tiles of rows the streams are the
// tiles, over the same blocks, so each K and V block loaded feeds 256 rows;
// with one tile left they take alternate blocks of it and are joined at the
// end.
//
// The running maximum is only raised when a row's new maximum is above it by
// more than 8 (in powers of two): P then stays below 2^8, within both types'
// range, sums are fp32, and O is rescaled in few blocks instead of all.  P is
// handed over in halves, so the product with V starts on the first.
//
// Bound by the tensor cores: a block and two tiles take 2048 clocks of
// products (N = 128: 64 clocks each), and QK^T reads shared memory at its full
// 128 bytes a clock.  Measured, 1024 rows over 128 Ki keys: 2570 clocks a block,
// 2410 with the softmax left out; 554 GFLOP in 350 us on the whole card, where
// its power limit holds plain products near 1.95 PFLOP/s.  Measured and
// dropped: steps of 64 keys with two S buffers a stream, which need not wait
// for S (470 us: products of N = 64 read Q twice as often); two threads a row
// (5 % slower); waits that poll without being suspended (6 % slower).
//
// Registers: 168 a thread at launch; the prompts' form spills 32 bytes, the
// shared prefix's none.
//
// Warps: 0-3 softmax of stream 0, 4-7 of stream 1 (a warp may reach only the
// 32 lanes of tensor memory its index modulo 4 names), 8 loads (one lane per
// TMA box), 9 the matrix products.  One persistent CTA an SM (all 512 columns
// of tensor memory); items of work are dealt in turn.
#include <algorithm>

#include "attn_tiles.cuh"

namespace qg {
namespace attn {
namespace {

constexpr int kWarpLoad = 8, kWarpMma = 9;
constexpr int kThreads = 384;                // warps 10 and 11 only fill the third warpgroup
// Registers of a thread: 168 at launch (65536 over 384), then shared out by
// warpgroup, 192 for the softmax's (a row of S, 128 values, in registers) and
// 120 for the other: 2 * 192 + 120 = 3 * 168.
constexpr int kRegsSoftmax = 192, kRegsOther = 120;
static_assert(2 * kRegsSoftmax + kRegsOther == 3 * 168, "registers shared out are those of the launch");

template <int D> struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr int HALF = 128 * 128;                 // bytes of 128 rows of 64 values
    static constexpr int TILE = HALVES * HALF;             // a Q tile, a K or a V block
    static constexpr int SLOTS = D == 128 ? 5 : 8;         // ring of K and V blocks
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_BAR = OFF_KV + SLOTS * TILE;
    static constexpr int OFF_ML = OFF_BAR + 256;           // (m, l) of stream 1's rows (joining)
    static constexpr int SMEM = OFF_ML + 128 * 8;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// Inclusive sums over the block's threads.
template <typename V>
__device__ __forceinline__ V block_sums(V v, V (&scratch)[32], V& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
        const V u = __shfl_up_sync(0xffffffffu, v, i);
        if (lane >= i) v += u;
    }
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    if (warp == 0) {
        V w = lane < (int)blockDim.x / 32 ? scratch[lane] : 0;
#pragma unroll
        for (int i = 1; i < 32; i *= 2) {
            const V u = __shfl_up_sync(0xffffffffu, w, i);
            if (lane >= i) w += u;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    total = scratch[31];
    if (warp) v += scratch[warp - 1];
    __syncthreads();
    return v;
}

// Lays the line of prompts out: one CTA, two runs of sums (pairs over the
// sequences, blocks over the pairs).
__global__ void __launch_bounds__(1024) k_attn_layout(const __grid_constant__ Args a, const __grid_constant__ Layout lay)
{
    __shared__ long long wide[32];
    __shared__ int scratch[32];
    __shared__ int longest;   // blocks of any pair
    if (threadIdx.x == 0) longest = 0;
    kv::pdl_wait();
    kv::pdl_release();
    const int per2 = 2 * lay.per;
    // Offsets that are not ascending may give every sequence all the tokens: 2^30 sequences of 2^22 pairs.  So the
    // pairs are summed in 64 bits, and what is past max_pairs, more than ascending offsets can make, is left out:
    // `first` stays ascending, so each pair kept lies within its sequence's tokens.
    long long sum = 0;
    for (int b0 = 0; b0 < a.bt.B; b0 += (int)blockDim.x) {
        const int b = b0 + (int)threadIdx.x;
        int t0 = 0, t1 = 0;
        if (b < a.bt.B && !kv::token_range(a.bt, b, t0, t1)) kv::report(a.status);
        const long long n = (t1 - t0 + per2 - 1) / per2;
        long long total;
        const long long upto = block_sums(n, wide, total);
        if (b < a.bt.B) lay.first[b] = (int)min(sum + upto - n, (long long)lay.max_pairs);
        sum += total;
    }
    const int pairs = (int)min(sum, (long long)lay.max_pairs);
    if (threadIdx.x == 0) {
        lay.first[a.bt.B] = pairs;
        if (sum > pairs) kv::report(a.status);
    }
    __syncthreads();
    const int np = (a.bt.prefix_len + KB - 1) / KB;
    int blocks = 0, total, most = 0;
    for (int i0 = 0; i0 < pairs; i0 += (int)blockDim.x) {
        const int i = i0 + (int)threadIdx.x;
        Pair p{0, 0, 0};
        int n = 0;
        if (i < pairs) {
            int hi = a.bt.B;   // the last sequence that starts at or before pair i
            while (hi - p.b > 1) {
                const int mid = (p.b + hi) / 2;
                if (lay.first[mid] <= i) p.b = mid;
                else hi = mid;
            }
            int t0, t1, len;
            kv::token_range(a.bt, p.b, t0, t1);
            if (!kv::own_length(a.bt, p.b, len)) kv::report(a.status);
            p.t0 = t0 + (i - lay.first[p.b]) * per2;
            const int own = len - (t1 - min(p.t0 + per2, t1));   // own tokens the pair's last token sees
            n = lay.extra + max(1, np + (max(0, own) + KB - 1) / KB);   // 1: a pair that sees nothing is still written
        }
        const int upto = block_sums(n, scratch, total);
        p.start = blocks + upto - n;
        if (i < pairs) lay.pair[i] = p;
        blocks += total;
        most = max(most, n);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) atomicMax(&longest, most);
    __syncthreads();
    // an item of n blocks touches at most ceil((n - 1) / run) + 1 runs
    const int run = max(max(kMinRun, (longest + kMostPieces - 2) / (kMostPieces - 1)),
                        (a.c.heads * blocks + lay.ctas - 1) / lay.ctas);
    if (threadIdx.x == 0) {
        lay.pair[pairs] = Pair{blocks, 0, 0};
        *lay.line = Line{run, blocks, pairs};
    }
    __syncthreads();
    for (int c = threadIdx.x; c < lay.ctas; c += (int)blockDim.x) {
        const int at = blocks ? c * run % blocks : 0;
        int lo = 0, hi = pairs;   // the pair the place lies in
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (lay.pair[mid].start <= at) lo = mid;
            else hi = mid;
        }
        lay.cut[c] = lo;
    }
}

template <typename T, int D, int KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tiles(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a,
                 const __grid_constant__ Deal deal, const __grid_constant__ Layout lay)
{
    using C = Cfg<D>;
    constexpr int NS = C::SLOTS, HALVES = C::HALVES;
    extern __shared__ __align__(1024) unsigned char smem[];   // the tiles' swizzle counts from 1024-byte boundaries
    const uint32_t sbase = ptx::smem_u32(smem), bars = sbase + C::OFF_BAR;
    const uint32_t q_full = bars, q_empty = bars + 8;
    auto s_full = [&](int s) { return bars + 16 + 8 * s; };     // S of stream s is in tensor memory
    auto p_full = [&](int s, int h) { return bars + 32 + 8 * (2 * s + h); };   // half h of P is, and O may be added to
    auto o_full = [&](int s) { return bars + 64 + 8 * s; };     // O is complete
    const uint32_t join_full = bars + 80, join_empty = bars + 88;   // stream 1's results for stream 0 to join: ready, read
    const uint32_t tail = bars + 96;      // a block of V with rows past the last key has arrived
    auto kv_full = [&](int x) { return bars + 104 + 8 * x; };
    auto kv_empty = [&](int x) { return bars + 104 + 8 * (NS + x); };
    const uint32_t products_done = bars + 104 + 16 * NS;   // when the CTA leaves
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 112 + 16 * NS);
    static_assert(112 + 16 * NS + 4 <= 256, "barriers");
    float2* ml1 = reinterpret_cast<float2*>(smem + C::OFF_ML);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 1);
        ptx::mbar_init(tail, 1);
        ptx::mbar_init(products_done, 1);
        for (int s = 0; s < 2; s++) {
            ptx::mbar_init(s_full(s), 1);
            ptx::mbar_init(p_full(s, 0), 4);
            ptx::mbar_init(p_full(s, 1), 4);
            ptx::mbar_init(o_full(s), 1);
        }
        ptx::mbar_init(join_full, 4);
        ptx::mbar_init(join_empty, 4);
        for (int x = 0; x < NS; x++) { ptx::mbar_init(kv_full(x), 1); ptx::mbar_init(kv_empty(x), 1); }
        ptx::fence_mbar_init();
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
    }
    if (warp == kWarpLoad && lane == 0) {
        ptx::prefetch_tensormap(&qmap);
        ptx::prefetch_tensormap(&kmap);
        ptx::prefetch_tensormap(&vmap);
    }
    kv::pdl_wait();
    kv::pdl_release();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // all columns are taken, so they start at 0, and the kernel's only shared memory starts at a multiple of its
    // alignment: known addresses let the products' operands be constants
    constexpr uint32_t tmem = 0;
    if (*tmem_slot != 0 || (sbase & 1023u)) {
        kv::report(a.status);
        __syncthreads();
        if (warp == kWarpMma) ptx::tmem_dealloc(*tmem_slot, kTmemCols);
        return;
    }
    bool ok = true;
    Item it;
    Cursor cur{(int)blockIdx.x, -1, 0};
    if constexpr (KEYS & kOwn) {
        const Line line = *lay.line;
        cur.i = (int)blockIdx.x * line.run;
        cur.head = line.head ? cur.i / line.head : 0;
        cur.pair = lay.cut[blockIdx.x];
    }
    const int per = (KEYS & kOwn) ? lay.per : deal.per;   // tokens of a tile

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kWarpLoad) {
            // ------------------------------------------------ loads
            const int boxes = KB / a.box_rows;                 // of a block, each rows of one page
            const int mine = lane % boxes, half = lane / boxes;
            const bool busy = half < HALVES;
            const int in_page_mask = (1 << a.c.page_shift) - 1;
            int pos = 0;                                       // loads so far
            int q_loaded = -1;                                 // phase of the last load of Q
            uint32_t item_phase = 0, tail_phase = 0;
            for (; ok && next_item<KEYS>(a, deal, lay, cur, it); item_phase ^= 1u) {
                const int n = it.blk1 - it.blk0;
                const int n_prefix = (it.prefix + in_page_mask) >> a.c.page_shift;
                const int* own_table = (KEYS & kOwn) ? a.bt.table + (long long)it.b * a.bt.table_ld : nullptr;
                auto keys_of = [&](int blk) { return blk < it.np ? min(KB, it.prefix - blk * KB) : max(0, min(KB, it.own - (blk - it.np) * KB)); };
                auto page_at = [&](int blk) -> int {
                    if (!busy || blk >= it.blk1 || mine * a.box_rows >= keys_of(blk)) return 0;
                    const int key = (blk < it.np ? blk : blk - it.np) * KB + mine * a.box_rows;
                    return blk < it.np ? page_of(a, a.bt.prefix_table, n_prefix, key >> a.c.page_shift)
                                       : page_of(a, own_table, a.bt.table_ld, key >> a.c.page_shift);
                };
                auto load = [&](bool is_v, int blk, int page) -> bool {
                    const int x = pos % NS, keys = keys_of(blk), used = (keys + a.box_rows - 1) / a.box_rows;
                    const uint32_t slot = C::OFF_KV + x * C::TILE;
                    if (!__all_sync(0xffffffffu, ptx::mbar_wait(kv_empty(x), ((pos / NS) & 1) ^ 1u))) return false;
                    pos++;
                    // V rows past the last key: what the page or an older block left there times 0 must be 0, so this warp waits
                    // for such a block itself and clears them
                    const bool ends = is_v && keys < KB;
                    const uint32_t bar = ends ? tail : kv_full(x);
                    if (lane == 0) ptx::mbar_expect_tx(bar, (uint32_t)(used * HALVES * a.box_rows * 128));
                    __syncwarp();
                    if (busy && mine < used) {
                        const int key = (blk < it.np ? blk : blk - it.np) * KB + mine * a.box_rows;
                        tma_load_4d(sbase + slot + half * C::HALF + mine * a.box_rows * 128, is_v ? &vmap : &kmap, half * 64,
                                    key & in_page_mask, it.head, page, bar);
                    }
                    if (ends) {
                        if (!__all_sync(0xffffffffu, ptx::mbar_wait(tail, tail_phase))) return false;
                        tail_phase ^= 1u;
                        for (int e = lane; e < (KB - keys) * 8 * HALVES; e += 32) {
                            const int row = keys + e / (8 * HALVES), c = e % (8 * HALVES);
                            *reinterpret_cast<uint4*>(smem + slot + (c / 8) * C::HALF + row * 128 + (c % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        ptx::fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(kv_full(x));
                    }
                    return true;
                };
                int page = page_at(it.blk0);
                if (n > 0) ok = load(false, it.blk0, page);
                if (!ok) break;
                // the last item's Q is no longer read
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(q_empty, item_phase ^ 1u));
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t bytes = (uint32_t)(per * a.group) * 128u * HALVES;
                    ptx::mbar_expect_tx(q_full, it.two ? 2 * bytes : bytes);
                    for (int s = 0; s < (it.two ? 2 : 1); s++)
                        for (int h = 0; h < HALVES; h++)
                            tma_load_3d(sbase + s * C::TILE + h * C::HALF, &qmap, 64 * h, it.head * a.group,
                                        it.t0 + s * per, q_full);
                }
                q_loaded = (int)item_phase;
                __syncwarp();
                for (int j = 1; ok && j <= n; j++) {
                    const int next = j < n ? page_at(it.blk0 + j) : 0;
                    if (j < n) ok = load(false, it.blk0 + j, next);
                    if (ok) ok = load(true, it.blk0 + j - 1, page);
                    page = next;
                }
            }
            // no copy is in flight when the CTA leaves, not even after a wait that gave up
            for (int i = max(0, pos - NS); i < pos; i++) ok = ptx::mbar_wait(kv_full(i % NS), (i / NS) & 1) && ok;
            if (q_loaded >= 0) ok = ptx::mbar_wait(q_full, (uint32_t)q_loaded) && ok;
        } else if (warp == kWarpMma && elect_lane()) {
            // ------------------------------------------------ matrix products, by one lane
            constexpr uint32_t id_qk = idesc<T>(KB, false), id_pv = idesc<T>(D, true);
            uint32_t item_phase = 0, p_phase[2] = {0, 0};
            int base = 0;   // ring position of the item's first load
            auto wait_kv = [&](int pos) { return ptx::mbar_wait(kv_full(pos % NS), (pos / NS) & 1); };
            auto release = [&](int pos) { commit(kv_empty(pos % NS)); };
            auto qk = [&](auto tile, auto s, int pos) {
                const uint32_t ad = desc_low(sbase + tile.value * C::TILE, 16);
                const uint32_t bd = desc_low(sbase + C::OFF_KV + (pos % NS) * C::TILE, 16);
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t off = (uint32_t)(((k / 4) * C::HALF + (k % 4) * 32) >> 4);
                    mma_ss(tmem + 128 * s.value, ad + off, bd + off, id_qk, k != 0);
                }
                commit(s_full(s.value));
            };
            // half h of P times half h of the V block
            auto pv = [&](auto s, auto h, int pos, bool first) {
                const uint32_t bd = desc_low(sbase + C::OFF_KV + (pos % NS) * C::TILE, C::HALF);
#pragma unroll
                for (int k = 4 * h.value; k < 4 * h.value + 4; k++)
                    mma_ts(tmem + kColO + 128 * s.value, tmem + 128 * s.value + 8 * k, bd + (uint32_t)((k * 2048) >> 4),
                           id_pv, k != 0 || !first);
            };
            auto wait_p = [&](int s, int h) {
                const bool r = ptx::mbar_wait(p_full(s, h), p_phase[s]);
                if (h) p_phase[s] ^= 1u;
                ptx::tc_fence_after();
                return r;
            };
            for (; ok && next_item<KEYS>(a, deal, lay, cur, it); item_phase ^= 1u) {
                const int n = it.blk1 - it.blk0;
                const int step = it.two ? 1 : 2;       // a stream's next block
                ok = ptx::mbar_wait(q_full, item_phase);
                // S of the streams' first blocks
                for (int j = 0; ok && j < min(step, n); j++) {
                    ok = wait_kv(base + pos_k(j));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (j == 0) qk(Const<0>{}, Const<0>{}, base + pos_k(j));
                    else qk(Const<0>{}, Const<1>{}, base + pos_k(j));
                    if (it.two) qk(Const<1>{}, Const<1>{}, base + pos_k(j));
                    release(base + pos_k(j));
                }
                if (n <= step) commit(q_empty);
                // one stream's turn in round j: its P of block j, then its S of block j + step
                auto turn = [&](auto tile, auto s, int j, bool last_use) {
                    const int v_pos = base + pos_v(j, n), k_pos = base + pos_k(j + step);
                    if (!(ok = ok && wait_p(s.value, 0))) return;
                    pv(s, Const<0>{}, v_pos, j < step);
                    if (!(ok = wait_p(s.value, 1))) return;
                    pv(s, Const<1>{}, v_pos, j < step);
                    if (j + step < n) {
                        qk(tile, s, k_pos);
                        if (last_use) {
                            release(k_pos);
                            if (j + step == n - 1) commit(q_empty);
                        }
                    } else {
                        commit(o_full(s.value));
                    }
                    if (last_use) release(v_pos);
                };
                for (int j = 0; ok && j < n; j++) {
                    // the loads of this round first: they have mostly arrived, and P has not
                    ok = wait_kv(base + pos_v(j, n)) && (j + step >= n || wait_kv(base + pos_k(j + step)));
                    if (it.two) {
                        turn(Const<0>{}, Const<0>{}, j, false);
                        turn(Const<1>{}, Const<1>{}, j, true);
                    } else if (j & 1) {
                        turn(Const<0>{}, Const<1>{}, j, true);
                    } else {
                        turn(Const<0>{}, Const<0>{}, j, true);
                    }
                }
                base += 2 * n;
            }
            // no product reads shared memory or writes tensor memory when the CTA leaves, not even after a wait that gave up
            commit(products_done);
            ok = ptx::mbar_wait(products_done, 0) && ok;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------ softmax, a row a thread
        const int s = warp / 4;
        const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16;
        const uint32_t t_s = tmem + lanes + 128 * s, t_o = tmem + lanes + kColO + 128 * s;
        const int r = 32 * (warp % 4) + lane;
        const int tok_in_tile = r / a.group;
        uint32_t s_phase = 0, o_phase = 0, join_phase = 0;
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
        while (ok && next_item<KEYS>(a, deal, lay, cur, it)) {
            const int n = it.blk1 - it.blk0, step = it.two ? 1 : 2;
            const int tok = it.t0 + (it.two ? s * per : 0) + tok_in_tile;
            const bool in = tok_in_tile < per && tok < it.t1;
            float m = -INFINITY, l = 0.0f;
            const int first = it.two ? 0 : s;
            for (int j = first; j < n; j += step) {
                const int blk = it.blk0 + j;
                const int vis = blk < it.np ? it.prefix - blk * KB : it.own0 + (tok - it.t0) - (blk - it.np) * KB;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full(s), s_phase));
                s_phase ^= 1u;
                if (!ok) break;
                ptx::tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; c++) tmem_ld32(t_s + 32 * c, x[c]);
                ptx::tmem_ld_wait();
                if (__any_sync(0xffffffffu, vis < KB)) {
#pragma unroll
                    for (int c = 0; c < 4; c++)
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            if (32 * c + e >= vis) x[c][e] = 0xFF800000u;   // -inf
                }
                float tm[8];   // independent maxima: no chain of 128
#pragma unroll
                for (int e = 0; e < 8; e++) tm[e] = __uint_as_float(x[0][e]);
#pragma unroll
                for (int c = 0; c < 4; c++)
#pragma unroll
                    for (int e = c == 0 ? 8 : 0; e < 32; e += 16)
#pragma unroll
                        for (int f = 0; f < 8; f++)
                            tm[f] = e + 8 + f < 32 ? fmaxf(fmaxf(tm[f], __uint_as_float(x[c][e + f])), __uint_as_float(x[c][(e + 8 + f) & 31]))
                                                   : fmaxf(tm[f], __uint_as_float(x[c][e + f]));
                float t = fmaxf(fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3])), fmaxf(fmaxf(tm[4], tm[5]), fmaxf(tm[6], tm[7])));
                t *= a.scale_log2;
                const bool raise = t > m + kRaise || (m == -INFINITY && t > -INFINITY);
                if (__any_sync(0xffffffffu, raise)) {
                    const float to = raise ? t : m;
                    const float f = to == m ? 1.0f : exp2_approx(m - to);
                    m = to;
                    l *= f;
                    if (j != first) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; c++) {
                            uint32_t o[32];
                            tmem_ld32(t_o + 32 * c, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(t_o + 32 * c, o);
                        }
                    }
                }
                const float u = m == -INFINITY ? 0.0f : m;   // a row that has seen nothing: all terms 2^-inf
                const float2 u2 = make_float2(-u, -u);
                float2 sum[4] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int h = 0; h < 2; h++) {   // in halves: the product with V starts on the first
#pragma unroll
                    for (int c = 2 * h; c < 2 * h + 2; c++) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const float2 y = fma2(make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])),
                                                  scale2, u2);
                            const float2 z = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            sum[e & 3] = add2(sum[e & 3], z);
                            p[e] = kv::pack2<T>(z.x, z.y);
                        }
                        tmem_st16(t_s + 16 * c, p);
                    }
                    tmem_st_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(p_full(s, h));
                }
                sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += sum[0].x + sum[0].y;
            }
            if (!ok) break;
            // ------------------------------------------------ the item's rows
            const bool ran = n > first;
            if (ran) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(o_full(s), o_phase));
                o_phase ^= 1u;
                if (!ok) break;
                ptx::tc_fence_after();
            }
            float w0 = 1.0f, w1 = 0.0f;       // weights of the two streams' O
            const bool both = !it.two && n > 1;
            if (!it.two) {
                if (s == 1) {
                    ml1[r] = make_float2(m, l);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(join_full);
                } else {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(join_full, join_phase));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const float2 v = ml1[r];
                    const float to = fmaxf(m, v.x), u = to == -INFINITY ? 0.0f : to;
                    w0 = exp2_approx(m - u);
                    w1 = exp2_approx(v.x - u);
                    l = l * w0 + v.y * w1;
                    m = to;
                }
            }
            if (it.two || s == 0) {
                const int hq = it.head * a.group + (r - tok_in_tile * a.group);
                const long long row = (long long)tok * a.heads_q + hq;
                const bool final = it.whole;
                const float inv = inverse(l);
                if (final) { w0 *= inv; w1 *= inv; }
                const long long at = (KEYS & kOwn) ? (long long)it.part * kSlotRows + (it.two ? 128 * s : 0) + r
                                                   : (long long)it.part * a.rows + row;
                if (in) {
                    if (final) store_lse(a, row, m, l);
                    else a.part_ml[at] = make_float2(m, l);
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; c++) {
                    uint32_t o[32];
                    if (ran) {
                        tmem_ld32(t_o + 32 * c, o);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * w0);
                        if (both) {
                            uint32_t o1[32];
                            tmem_ld32(t_o + 128 + 32 * c, o1);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; e++)
                                o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e])));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e++) o[e] = 0u;
                    }
                    if (!in) continue;
                    if (!final) {
                        if (l != 0.0f)
#pragma unroll
                            for (int e = 0; e < 32; e += 8) store32(a.part_o + at * D + 32 * c + e, o + e);
                    } else {
                        const long long to = tok * a.ldo + (long long)hq * D + 32 * c;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) store_out8(a, to + e, o + e);
                    }
                }
            }
            if (!it.two) {
                if (s == 0) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(join_empty);
                } else {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(join_empty, join_phase));
                    ptx::tc_fence_after();
                }
                join_phase ^= 1u;
            }
        }
    }
    if (!ok && a.status) atomicExch(a.status, (int)QG_ERR_TIMEOUT);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWarpMma) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <typename T, int D, int KEYS>
cudaError_t launch_one(const Args& a, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                       const Deal& d, const Layout& lay, int ctas, cudaStream_t s)
{
    auto kernel = k_attn_tiles<T, D, KEYS>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = kv::allow_smem(kernel, Cfg<D>::SMEM, done);
    if (e != cudaSuccess) return e;
    return kv::launch_dependent(kernel, dim3((unsigned)ctas), kThreads, Cfg<D>::SMEM, s, qmap, kmap, vmap, a, d, lay);
}

template <int KEYS>
cudaError_t by_type(const Args& a, int dtype, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                    const Deal& d, const Layout& lay, int ctas, cudaStream_t s)
{
    if (dtype == QG_T_BF16)
        return a.c.dim == 128 ? launch_one<__nv_bfloat16, 128, KEYS>(a, qmap, kmap, vmap, d, lay, ctas, s)
                              : launch_one<__nv_bfloat16, 64, KEYS>(a, qmap, kmap, vmap, d, lay, ctas, s);
    return a.c.dim == 128 ? launch_one<__half, 128, KEYS>(a, qmap, kmap, vmap, d, lay, ctas, s)
                          : launch_one<__half, 64, KEYS>(a, qmap, kmap, vmap, d, lay, ctas, s);
}

}  // namespace

cudaError_t launch_layout(const Args& a, const Layout& lay, cudaStream_t s)
{
    return kv::launch_dependent(k_attn_layout, dim3(1), 1024, 0, s, a, lay);
}

cudaError_t launch_tiles_shared(const Args& a, int dtype, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, const Deal& d, int ctas, cudaStream_t s)
{
    return by_type<kPrefix>(a, dtype, qmap, kmap, vmap, d, Layout{}, std::min(ctas, d.slots()), s);
}

cudaError_t launch_tiles(const Args& a, int dtype, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, const Layout& lay, cudaStream_t s)
{
    const cudaError_t e = launch_layout(a, lay, s);
    if (e != cudaSuccess) return e;
    return by_type<kPrefix | kOwn>(a, dtype, qmap, kmap, vmap, Deal{}, lay, lay.ctas, s);
}

}  // namespace attn
}  // namespace qg
