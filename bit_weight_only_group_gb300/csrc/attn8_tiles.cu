// Attention over the 8-bit cache for many query rows per key/value head, on the
// 5th-generation tensor cores: the tile kernel of attn_tiles.cu (128 rows a tile,
// blocks of 128 keys, two streams, P back through tensor memory, the work dealt
// the same way) with codes in place of 16-bit values.
//
// The tensor core takes fp16.  Four warps copy codes from their pages to places
// of their own in shared memory (asynchronously, two blocks ahead: a thread reads
// only what it copied), turn them into fp16, two an instruction, and store them
// where TMA would have put the 16-bit block; a block and its conversion serve
// both tiles (256 rows).  A warp has two runs of 16 keys of each K or V block,
// each in one page.  (Loaded into registers, where one block at a time has room,
// a block took its latency and its conversion one after the other: 128 rows over
// 128 Ki keys 540 us.)  The softmax's warps scale the rows of q by powers of two
// and store them as fp16 before they write an item's results, so that S of the
// next is there when they have.
// The scales do not touch the operands: the softmax multiplies the logits of 16
// keys by the K scale (in the fused product that its argument takes anyway) and
// adds the V scale's exponent to that argument (attn.cuh), so an element costs
// what it costs with 16-bit values, and a group of 16 a few operations more.
//
// fp8 products would take Q and P in several E4M3 parts (two hold bf16's 8
// bits): the same tensor-core time as fp16, while P's split costs the softmax
// four conversions a pair, which run at 16 to 32 a clock (measured: 21 to E4M3).
//
// Warps: 0-3 softmax of stream 0, 4-7 of stream 1, 8-11 codes, 12 the products, 13
// looks the scales up and leaves them in shared memory (14 and 15 only fill the
// fourth warpgroup).
#include <algorithm>

#include "attn_tiles.cuh"

namespace qg {
namespace attn {
namespace {

constexpr int kWarpConvert = 8, kWarpMma = 12, kWarpScales = 13;
constexpr int kThreads = 512;
// Registers of a thread: 128 at launch (65536 over 512), then shared out by warpgroup.
constexpr int kRegsLaunch = 128, kRegsSoftmax = 192, kRegsConvert = 80, kRegsMma = 48;
static_assert(2 * kRegsSoftmax + kRegsConvert + kRegsMma == 4 * kRegsLaunch, "registers shared out are those of the launch");

// Scales of a block: the K scales of its 16s of keys, the V scales' exponents, and those scales' reciprocals.
constexpr int kScales = 24, kScaleSlots = 4;

template <int D> struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr int HALF = 128 * 128;                 // bytes of 128 rows of 64 values
    static constexpr int TILE = HALVES * HALF;             // a Q tile, a K or a V block, in fp16
    static constexpr int SLOTS = D == 128 ? 4 : 8;         // ring of K and V blocks
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int RAW = KB * D, RAWS = D == 128 ? 2 : 4;   // a block's codes, and blocks in flight
    static constexpr int OFF_RAW = OFF_KV + SLOTS * TILE;
    static constexpr int OFF_BAR = OFF_RAW + RAWS * RAW;
    static constexpr int OFF_ML = OFF_BAR + 512;           // (m, l) of stream 1's rows (joining)
    static constexpr int OFF_BACK = OFF_ML + 128 * 8;      // what stream 0 scaled its rows of Q by, for stream 1
    static constexpr int OFF_SCALES = OFF_BACK + 2 * 128;  // of each stream's next blocks
    static constexpr int SMEM = OFF_SCALES + 2 * kScaleSlots * kScales * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    // 16 keys of a converting warp: LANES lanes a key with 16 codes each, CHUNKS times ROWS keys
    static constexpr int LANES = D / 16, ROWS = 32 / LANES, CHUNKS = 16 / ROWS;
};

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <int D, int KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn8_tiles(const __grid_constant__ Args8 p8, const __grid_constant__ Deal deal, const __grid_constant__ Layout lay)
{
    using C = Cfg<D>;
    constexpr int NS = C::SLOTS;
    const Args& a = p8.a;
    extern __shared__ __align__(1024) unsigned char smem[];   // the tiles' swizzle counts from 1024-byte boundaries
    const uint32_t sbase = ptx::smem_u32(smem), bars = sbase + C::OFF_BAR;
    const uint32_t q_full = bars, q_empty = bars + 8;
    auto s_full = [&](int s) { return bars + 16 + 8 * s; };     // S of stream s is in tensor memory
    auto p_full = [&](int s, int h) { return bars + 32 + 8 * (2 * s + h); };   // half h of P is, and O may be added to
    auto o_full = [&](int s) { return bars + 64 + 8 * s; };     // O is complete
    const uint32_t join_full = bars + 80, join_empty = bars + 88;   // stream 1's results for stream 0 to join: ready, read
    auto kv_full = [&](int x) { return bars + 96 + 8 * x; };
    auto kv_empty = [&](int x) { return bars + 96 + 8 * (NS + x); };
    const uint32_t products_done = bars + 96 + 16 * NS;   // when the CTA leaves
    auto back_full = [&](int x) { return bars + 104 + 16 * NS + 8 * x; };   // a single tile's scalings are in shared memory
    auto scale_full = [&](int s, int x) { return bars + 120 + 16 * NS + 8 * (kScaleSlots * s + x); };
    auto scale_empty = [&](int s, int x) { return bars + 120 + 16 * NS + 8 * (kScaleSlots * (2 + s) + x); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 120 + 16 * NS + 32 * kScaleSlots);
    static_assert(120 + 16 * NS + 32 * kScaleSlots + 4 <= 512, "barriers");
    float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALES);
    float2* ml1 = reinterpret_cast<float2*>(smem + C::OFF_ML);
    signed char* back0 = reinterpret_cast<signed char*>(smem + C::OFF_BACK);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        ptx::mbar_init(q_full, 8);
        ptx::mbar_init(q_empty, 1);
        ptx::mbar_init(products_done, 1);
        for (int s = 0; s < 2; s++) {
            ptx::mbar_init(s_full(s), 1);
            ptx::mbar_init(p_full(s, 0), 4);
            ptx::mbar_init(p_full(s, 1), 4);
            ptx::mbar_init(o_full(s), 1);
            ptx::mbar_init(back_full(s), 4);
            for (int x = 0; x < kScaleSlots; x++) { ptx::mbar_init(scale_full(s, x), 1); ptx::mbar_init(scale_empty(s, x), 4); }
        }
        ptx::mbar_init(join_full, 4);
        ptx::mbar_init(join_empty, 4);
        for (int x = 0; x < NS; x++) { ptx::mbar_init(kv_full(x), 4); ptx::mbar_init(kv_empty(x), 1); }
        ptx::fence_mbar_init();
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
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
    Item it{};
    Cursor cur{(int)blockIdx.x, -1, 0};
    if constexpr (KEYS & kOwn) {
        const Line line = *lay.line;
        cur.i = (int)blockIdx.x * line.run;
        cur.head = line.head ? cur.i / line.head : 0;
        cur.pair = lay.cut[blockIdx.x];
    }
    const int per = (KEYS & kOwn) ? lay.per : deal.per;   // tokens of a tile
    const int in_page_mask = (1 << a.c.page_shift) - 1;

    // Keys of a block of an item that any row sees, the first key's place, and the table's entry for 16 of them.
    auto keys_of = [&](const Item& it, int blk) { return blk < it.np ? min(KB, it.prefix - blk * KB) : max(0, min(KB, it.own - (blk - it.np) * KB)); };
    auto key_of = [&](const Item& it, int blk, int group) { return (blk < it.np ? blk : blk - it.np) * KB + 16 * group; };
    auto entry_at = [&](const Item& it, int blk, int group) {
        const bool there = blk < it.blk1 && 16 * group < keys_of(it, blk);
        const int* table = !(KEYS & kOwn) || blk < it.np ? a.bt.prefix_table : a.bt.table + (long long)it.b * a.bt.table_ld;
        return table_entry(a, table, key_of(it, blk, group) >> a.c.page_shift, there);
    };

    if (warp >= kWarpMma) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
        if (warp == kWarpMma && elect_lane()) {
            // ------------------------------------------------ matrix products, by one lane
            constexpr uint32_t id_qk = idesc<__half>(KB, false), id_pv = idesc<__half>(D, true);
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
        if (warp == kWarpScales) {
            // ------------------------------------------------ scales: lanes 0-7 K, 8-15 the exponents of V, 16-23 reciprocals
            const int group = lane % 8;
            int slot[2] = {0, 0};
            uint32_t round[2] = {1, 1};
            while (ok && next_item<KEYS>(a, deal, lay, cur, it)) {
                const int n = it.blk1 - it.blk0;
                auto byte_at = [&](const Entry& e, int blk) {
                    return scale_byte(p8, lane >= 8, checked_page(a, e), (key_of(it, blk, group) & in_page_mask) / 16, it.head);
                };
                // the table's entries two blocks ahead, scales one
                Entry next = entry_at(it, it.blk0 + 1, group);
                int byte = byte_at(entry_at(it, it.blk0, group), it.blk0);
                for (int j = 0; ok && j < n; j++) {
                    const int e = scale_exp(byte);
                    byte = byte_at(next, it.blk0 + j + 1);
                    next = entry_at(it, it.blk0 + j + 2, group);
                    const float f = lane < 8 ? kv8::pow2(e) : lane < 16 ? (float)e : kv8::pow2(-e);
                    for (int s = it.two ? 0 : j & 1; ok && s < (it.two ? 2 : (j & 1) + 1); s++) {
                        const int x = slot[s & 1];
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(scale_empty(s, x), round[s & 1]));
                        if (!ok) break;
                        if (lane < kScales) scales[(s * kScaleSlots + x) * kScales + lane] = f;
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(scale_full(s, x));
                        if (++slot[s & 1] == kScaleSlots) { slot[s & 1] = 0; round[s & 1] ^= 1u; }
                    }
                }
            }
        }
    } else if (warp >= kWarpConvert) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
        // ------------------------------------------------ codes to fp16: keys 16 w .. and 16 (w + 4) .. of a block
        // keys row0 + c ROWS, codes 16 chunk ..: eight lanes take two rows' half of 64 values, so that their stores meet all banks
        const int w = warp - kWarpConvert, chunk = lane % 4 + (D == 128 ? lane / 8 % 2 * 4 : 0);
        const int row0 = D == 128 ? lane / 4 % 2 + lane / 16 * 2 : lane / 4;
        uint32_t to[2];   // of rows row0 + c ROWS for even, odd c
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const int row = row0 + c * C::ROWS;
            to[c] = (uint32_t)(chunk / 4 * C::HALF + (16 * w + row) * 128 + 16 * (2 * (chunk % 4) ^ (row & 7)));
        }
        const int group = w + 4 * (lane & 1);   // the keys whose page this lane looks up
        const long long hop = (long long)C::ROWS * a.c.token_stride;
        const uint32_t raw = sbase + C::OFF_RAW + 16 * (threadIdx.x - 32 * kWarpConvert);   // this thread's places
        int slot = 0, raw_slot = 0;
        uint32_t round = 1;   // parity of the wait for a free slot
        while (ok && next_item<KEYS>(a, deal, lay, cur, it)) {
            const int n = it.blk1 - it.blk0, loads = 2 * n;
            const long long mine = (long long)it.head * a.c.head_stride + (long long)row0 * a.c.token_stride + 16 * chunk;
            // where this lane's 16 keys of a block begin among the codes: of the last block K was loaded for, and the one before;
            // -1: nothing there to load.  The next one's entry of the table is on its way.
            long long now = -1, before = -1;
            Entry entry = entry_at(it, it.blk0, group);
            // load number i, in the order K0, K1 V0, K2 V1, ..
            struct Load { const uint8_t* from; long long at; int left; };   // left: keys of the block
            auto next_load = [&](int i) -> Load {
                const bool v = i != 0 && (!(i & 1) || i == loads - 1);
                const int blk = it.blk0 + (i == loads - 1 ? n - 1 : i == 0 ? 0 : i & 1 ? (i + 1) / 2 : i / 2 - 1);
                if (!v) {
                    const int page = checked_page(a, entry);
                    before = now;
                    now = page >= 0 && page < a.c.num_pages
                              ? (long long)page * a.c.page_stride + (long long)(key_of(it, blk, group) & in_page_mask) * a.c.token_stride : -1;
                    entry = entry_at(it, blk + 1, group);
                }
                return Load{v ? p8.v_codes : p8.k_codes, !v || i == loads - 1 ? now : before, keys_of(it, blk)};
            };
            // a load's codes to this thread's places of a raw block: keys past the last, and pages not to be followed, are zeros
            auto fetch = [&](int i) {
                if (i < loads) {
                    const Load l = next_load(i);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const long long at = __shfl_sync(0xffffffffu, l.at, h);
                        const uint8_t* p = at >= 0 ? l.from + at + mine : l.from;
#pragma unroll
                        for (int c = 0; c < C::CHUNKS; c++) {
                            const bool there = at >= 0 && 16 * w + row0 + 64 * h + c * C::ROWS < l.left;
                            copy16(raw + raw_slot * C::RAW + (h * C::CHUNKS + c) * (128 * 16), there ? p + c * hop : l.from, there);
                        }
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (++raw_slot == C::RAWS) raw_slot = 0;
            };
            raw_slot = 0;
#pragma unroll 1
            for (int d = 0; d < C::RAWS; d++) fetch(d);
#pragma unroll 1
            for (int i = 0; i < loads; i++) {
                asm volatile("cp.async.wait_group %0;" ::"n"(C::RAWS - 1) : "memory");
                uint4 r[2 * C::CHUNKS];
#pragma unroll
                for (int c = 0; c < 2 * C::CHUNKS; c++)
                    r[c] = *reinterpret_cast<const uint4*>(smem + C::OFF_RAW + raw_slot * C::RAW + c * (128 * 16) + 16 * (threadIdx.x - 32 * kWarpConvert));
                fetch(i + C::RAWS);   // over what has just been read
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(kv_empty(slot), round));
                if (!ok) break;
                unsigned char* into = smem + C::OFF_KV + slot * C::TILE;
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int c = 0; c < C::CHUNKS; c++) {
                        const uint4 x = r[h * C::CHUNKS + c];
                        const uint32_t at = to[c & 1] + (64 * h + (c & ~1) * C::ROWS) * 128;
                        *reinterpret_cast<uint4*>(into + at) =
                            make_uint4(kv8::decode_lo(x.x), kv8::decode_hi(x.x), kv8::decode_lo(x.y), kv8::decode_hi(x.y));
                        *reinterpret_cast<uint4*>(into + (at ^ 16)) =
                            make_uint4(kv8::decode_lo(x.z), kv8::decode_hi(x.z), kv8::decode_lo(x.w), kv8::decode_hi(x.w));
                    }
                ptx::fence_proxy_async();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(kv_full(slot));
                if (++slot == NS) { slot = 0; round ^= 1u; }
            }
            // no copy is in flight when the CTA leaves, or where the next item's go
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------ softmax, a row a thread
        const int s = warp / 4;
        const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16;
        const uint32_t t_s = tmem + lanes + 128 * s, t_o = tmem + lanes + kColO + 128 * s;
        const int r = 32 * (warp % 4) + lane;
        const int tok_in_tile = r / a.group;
        uint32_t s_phase = 0, o_phase = 0, join_phase = 0, item_phase = 0;
        int slot = 0;          // of the scales
        uint32_t round = 0;
        int singles = 0;   // items of a single tile
        // The warp's 32 rows of an item's Q to shared memory, each scaled by 2^-back: the exponent of this lane's row.  Done
        // before the last item's results are written, so that S of the new item is there when they are.
        auto prepare = [&](const Item& it) -> int {
            int back = 0;
            if (it.two || s == 0) {
                constexpr int QL = D / 8, QROWS = 32 / QL, QN = 32 / QROWS;   // lanes of a row, rows at a time, times
                const int qr = lane / QL, qc = lane % QL;
                const bool bf = p8.q_type == QG_T_BF16;
                uint4 w[QN];
#pragma unroll
                for (int i = 0; i < QN; i++) {
                    const int row = 32 * (warp % 4) + i * QROWS + qr, t = row / a.group, at = it.t0 + s * per + t;
                    w[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (t < per && at < it.t1)
                        w[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at * a.ldq +
                                                                    (long long)(it.head * a.group + row % a.group) * D) + qc);
                }
                // the last item's Q is no longer read
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(q_empty, item_phase ^ 1u));
                if (!ok) return 0;
#pragma unroll
                for (int i = 0; i < QN; i++) {
                    const int row = 32 * (warp % 4) + i * QROWS + qr;
                    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    float2 f[4];
                    float amax = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        f[e] = bf ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e])) : kv8::half2_floats(u[e]);
                        amax = fmaxf(amax, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
                    }
#pragma unroll
                    for (int e = QL / 2; e > 0; e /= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, e));
                    const int ex = row_exp(amax);
                    const float up = kv8::pow2(14 - ex);
                    const int of = __shfl_sync(0xffffffffu, ex - 14, lane % QROWS * QL);   // of row i QROWS + lane % QROWS
                    if (lane / QROWS == i) back = of;
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) h[e] = kv::pack2<__half>(f[e].x * up, f[e].y * up);
                    *reinterpret_cast<uint4*>(smem + s * C::TILE + qc / 8 * C::HALF + row * 128 + 16 * (qc % 8 ^ (row & 7))) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
                ptx::fence_proxy_async();
            }
            item_phase ^= 1u;
            // both streams work on a single tile's rows: stream 0 leaves the exponents in one of two buffers, each written again
            // only after the streams have met at the end of its item
            signed char* shared = back0 + 128 * (singles & 1);
            if (!it.two && s == 0) shared[r] = (signed char)back;
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(q_full);
                if (!it.two && s == 0) ptx::mbar_arrive(back_full(singles & 1));
            }
            if (!it.two && s == 1) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(back_full(singles & 1), (singles >> 1) & 1));
                back = shared[r];
            }
            if (!it.two) singles++;
            return back;
        };
        bool more = next_item<KEYS>(a, deal, lay, cur, it);
        int back = more ? prepare(it) : 0;
        while (ok && more) {
            const int n = it.blk1 - it.blk0, step = it.two ? 1 : 2;
            const int tok = it.t0 + (it.two ? s * per : 0) + tok_in_tile;
            const bool in = tok_in_tile < per && tok < it.t1;
            float m = -INFINITY, l = 0.0f;
            const int first = it.two ? 0 : s;
            const float row_scale = a.scale_log2 * kv8::pow2(back);
            // what the logits of 16 keys are multiplied by: at least the smallest normal number, since a masked logit times 0
            // would be a NaN
            auto factor = [&](float scale) { return fmaxf(row_scale * scale, 1.17549435e-38f); };
            for (int j = first; j < n; j += step) {
                const int blk = it.blk0 + j;
                const int vis = blk < it.np ? it.prefix - blk * KB : it.own0 + (tok - it.t0) - (blk - it.np) * KB;
                const float* sc = scales + (s * kScaleSlots + slot) * kScales;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(scale_full(s, slot), round));
                if (!ok) break;
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
                float t = -INFINITY;   // the largest s + ev
#pragma unroll
                for (int g = 0; g < 8; g++) {
                    const uint32_t* y = x[g / 2] + 16 * (g % 2);
                    float u = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1])), v = fmaxf(__uint_as_float(y[2]), __uint_as_float(y[3]));
#pragma unroll
                    for (int e = 4; e < 16; e += 4) {
                        u = fmaxf(fmaxf(u, __uint_as_float(y[e])), __uint_as_float(y[e + 1]));
                        v = fmaxf(fmaxf(v, __uint_as_float(y[e + 2])), __uint_as_float(y[e + 3]));
                    }
                    t = fmaxf(t, fmaf(fmaxf(u, v), factor(sc[g]), sc[8 + g]));
                }
                const bool raise = t > m + kRaise || (m == -INFINITY && t > -INFINITY);
                if (__any_sync(0xffffffffu, raise)) {
                    const float to = raise ? t : m;
                    const float w = to == m ? 1.0f : exp2_approx(m - to);
                    m = to;
                    l *= w;
                    if (j != first) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; c++) {
                            uint32_t o[32];
                            tmem_ld32(t_o + 32 * c, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * w);
                            tmem_st32(t_o + 32 * c, o);
                        }
                    }
                }
                const float u = m == -INFINITY ? 0.0f : m;   // a row that has seen nothing: all terms 2^-inf
#pragma unroll
                for (int h = 0; h < 2; h++) {   // in halves: the product with V starts on the first
#pragma unroll
                    for (int c = 2 * h; c < 2 * h + 2; c++) {
                        uint32_t p[16];
#pragma unroll
                        for (int q = 0; q < 2; q++) {
                            const int g = 2 * c + q;
                            const float f = factor(sc[g]), add = sc[8 + g] - u;
                            const float2 f2 = make_float2(f, f), c2 = make_float2(add, add);
                            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                            for (int e = 8 * q; e < 8 * q + 8; e++) {
                                const float2 y = fma2(make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), f2, c2);
                                const float2 z = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                                sum[e & 1] = add2(sum[e & 1], z);
                                p[e] = kv::pack2<__half>(z.x, z.y);
                            }
                            sum[0] = add2(sum[0], sum[1]);
                            l = fmaf(sum[0].x + sum[0].y, sc[16 + g], l);
                        }
                        tmem_st16(t_s + 16 * c, p);
                    }
                    tmem_st_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(p_full(s, h));
                }
                if (lane == 0) ptx::mbar_arrive(scale_empty(s, slot));
                if (++slot == kScaleSlots) { slot = 0; round ^= 1u; }
            }
            if (!ok) break;
            Item next;
            more = next_item<KEYS>(a, deal, lay, cur, next);
            if (more) back = prepare(next);
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
            it = next;
        }
    }
    if (!ok && a.status) atomicExch(a.status, (int)QG_ERR_TIMEOUT);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWarpMma) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int D, int KEYS>
cudaError_t launch_one(const Args8& p, const Deal& d, const Layout& lay, int ctas, cudaStream_t s)
{
    auto kernel = k_attn8_tiles<D, KEYS>;
    static std::atomic<unsigned long long> done{0};
    const unsigned long long ctx = current_context_id();
    if (!ctx || done.load(std::memory_order_acquire) != ctx) {
        // the warpgroups share out the registers of the launch: with any other number one would wait for ever
        cudaFuncAttributes at;
        cudaError_t e = cudaFuncGetAttributes(&at, kernel);
        if (e != cudaSuccess) return e;
        if (at.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        done.store(ctx, std::memory_order_release);
    }
    return kv::launch_dependent(kernel, dim3((unsigned)ctas), kThreads, Cfg<D>::SMEM, s, p, d, lay);
}

}  // namespace

cudaError_t launch_tiles8_shared(const Args8& p, const Deal& d, int ctas, cudaStream_t s)
{
    const int n = std::min(ctas, d.slots());
    return p.a.c.dim == 128 ? launch_one<128, kPrefix>(p, d, Layout{}, n, s) : launch_one<64, kPrefix>(p, d, Layout{}, n, s);
}

cudaError_t launch_tiles8(const Args8& p, const Layout& lay, cudaStream_t s)
{
    return p.a.c.dim == 128 ? launch_one<128, kPrefix | kOwn>(p, Deal{}, lay, lay.ctas, s)
                            : launch_one<64, kPrefix | kOwn>(p, Deal{}, lay, lay.ctas, s);
}

}  // namespace attn
}  // namespace qg
