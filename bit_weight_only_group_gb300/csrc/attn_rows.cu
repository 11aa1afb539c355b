// Attention for few query rows per key/value head: a decoding step's own
// tokens, 1 to 64 rows (tokens x query heads of one key/value head) a CTA.
//
// The keys are the bound: at R rows a key/value pair of 4 dim bytes takes
// 4 R dim operations, below the tensor cores' rate for R up to a few hundred.
// So K and V stream through shared memory once, by TMA (64 keys a stage, the
// page's place looked up by one lane per box), and warp-level matrix
// instructions (m16n8k16) do the products from there:
//     S = Q K^T      Q in registers as the A operand, 16 rows a warp
//     P = 2^(S scale_log2 - m), with the running maximum m and sum l
//     O = O 2^(m_old - m) + P V
// P goes from S's accumulator layout to the A operand's without leaving the
// thread.  Four warps split a stage's keys among them and the rows in blocks of
// 16 (RW row blocks x 4 / RW key ranges); each keeps m, l and O of its own
// keys, and the CTA joins them at the end.
//
// m, l and O are fp32.  P is rounded to the cache's type for the product with
// V, whose operands have 16 bits; to keep the rest of P would take a second
// product with V (half as many products again), which neither this kernel's
// warps nor the tensor-bound tile kernel have time for.  l is the sum before
// the rounding.  A probability is off by up to 2^-8 of itself in bf16, 2^-11 in
// fp16, either way, and the errors average over the keys: measured with fp32
// output against 64 bits, 5.4e-5 rms where the outputs are 0.047 rms (bf16, 16
// sequences over 4096 + 512 keys; rounding right outputs to bf16 alone is
// 7.8e-5), and 0.75e-5 of 0.039 (fp16, 48 sequences of up to 5 tokens;
// 0.81e-5).
#include <algorithm>

#include "attn.cuh"

namespace qg {
namespace attn {
namespace {

constexpr int KT = 64;                       // keys of a stage
constexpr int kWarps = 4;                    // consumer warps; warp 4 issues the loads
constexpr int kThreads = (kWarps + 1) * 32;

template <int D> struct Cfg {
    // stages in flight: with 128-wide heads two CTAs an SM (registers) and three stages of 32 KB each stream 6.3 TB/s,
    // three CTAs of two stages (128 registers, a few spilled) 5.6; with 64-wide heads three CTAs of four 16 KB stages.
    // At 168 registers (128-wide) and 128 (64-wide) the forms of 16 rows spill nothing, those of 32 rows 8 bytes (128-
    // wide), those of 64 rows 52 (prefix and own tokens in one launch 40 to 96) and 16 to 48 bytes a thread.
    static constexpr int MAX_STAGES = D == 128 ? 3 : 4;
    static constexpr int TILE = KT * D * 2;              // bytes of a K or V tile: per box [dim / 64][key][64 values], swizzled
    static constexpr int STAGE = 2 * TILE;
    static constexpr int OFF_ML = 2 * 8 * MAX_STAGES;    // after the barriers: (m, l) of the joining warps' rows
    static constexpr int REST = OFF_ML + kWarps * 16 * 8 + 1024;   // barriers, (m, l), alignment
    // the joining buffers (2 slots of 16 x D fp32) lie over the stages
    static_assert(2 * 16 * D * 4 <= STAGE, "joining buffers fit the stages");
};

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

template <int KEYS>
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
    it.np = (it.prefix + KT - 1) / KT;
    const int tiles = it.rows > 0 ? it.np + (it.own + KT - 1) / KT : 0;
    const int per = max(least_tiles, (tiles + parts - 1) / parts);
    it.tile0 = min(part * per, tiles);
    it.tile1 = min(it.tile0 + per, tiles);
    return it;
}

// The CTA numbered x of a launch's (unit, row block, part, head) CTAs.
struct Split {
    int part0, parts, least_tiles, row_blocks;
};

template <typename T, int D, int RW, int KEYS>
__device__ __forceinline__ void work(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& a, const Split& sp, int x,
                                     int stages, bool beside)
{
    using C = Cfg<D>;
    constexpr int KW = kWarps / RW, NK = KT / KW, HALVES = D / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem), bars = sbase + stages * C::STAGE;
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (C::MAX_STAGES + s); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // neighbouring CTAs take the heads of one unit (their rows of a page lie together when tokens come first)
    const int head = x % a.c.heads;
    x /= a.c.heads;
    const int part = x % sp.parts;
    x /= sp.parts;
    const int row_block = x % sp.row_blocks, unit = x / sp.row_blocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; s++) { ptx::mbar_init(full(s), 1); ptx::mbar_init(empty(s), kWarps); }
        ptx::fence_mbar_init();
    }
    if (warp == kWarps && lane == 0) { ptx::prefetch_tensormap(&kmap); ptx::prefetch_tensormap(&vmap); }
    __syncthreads();
    // beside: the kernel ahead writes nothing this one reads or writes, and started only after everything before it
    // had finished; then one CTA alone waits for it, so that this kernel does not finish first
    if (!beside) kv::pdl_wait();
    kv::pdl_release();
    if (beside && blockIdx.x == gridDim.x - 1) kv::pdl_wait();
    const Item it = find_item<KEYS>(a, unit, row_block, part, sp.parts, sp.least_tiles, 16 * RW, threadIdx.x == 0);
    if (it.rows == 0) return;
    bool ok = true;
    // keys of tile j that any row sees
    auto tile_keys = [&](int j) { return j < it.np ? min(KT, it.prefix - j * KT) : min(KT, it.own - (j - it.np) * KT); };

    if (warp == kWarps) {
        // ------------------------------------------------ loads: one lane per box
        const int boxes = KT / a.box_rows;                       // key ranges of a tile, each a page's rows
        const int mine = lane % boxes, is_v = lane / boxes;
        const bool busy = is_v < 2;
        const int* own_table = (KEYS & kOwn) ? a.bt.table + (long long)it.b * a.bt.table_ld : nullptr;
        const int n_prefix = (it.prefix + (1 << a.c.page_shift) - 1) >> a.c.page_shift;
        auto page_at = [&](int j) -> int {   // page of this lane's box of tile j
            if (!busy || j >= it.tile1 || mine * a.box_rows >= tile_keys(j)) return 0;
            const int key = (j < it.np ? j : j - it.np) * KT + mine * a.box_rows;
            return j < it.np ? page_of(a, a.bt.prefix_table, n_prefix, key >> a.c.page_shift)
                             : page_of(a, own_table, a.bt.table_ld, key >> a.c.page_shift);
        };
        int s = 0, issued = 0;
        uint32_t ph = 0;
        int page = page_at(it.tile0);
        for (int j = it.tile0; j < it.tile1; j++) {
            const int next = page_at(j + 1);
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(empty(s), ph ^ 1u));
            if (!ok) break;
            const int used = (tile_keys(j) + a.box_rows - 1) / a.box_rows;
            if (lane == 0) ptx::mbar_expect_tx(full(s), (uint32_t)(used * a.box_rows * (4 * D)));
            __syncwarp();
            if (busy && mine < used) {
                const int key = (j < it.np ? j : j - it.np) * KT + mine * a.box_rows;
                tma_load_5d(sbase + s * C::STAGE + is_v * C::TILE + mine * a.box_rows * (2 * D), is_v ? &vmap : &kmap, 0,
                            key & ((1 << a.c.page_shift) - 1), 0, head, page, full(s));
            }
            page = next;
            issued++;
            if (++s == stages) { s = 0; ph ^= 1u; }
        }
        // no copy is in flight when the CTA leaves, not even after a wait that gave up
        for (int i = min(stages, issued); i > 0; i--) {
            if (s-- == 0) { s = stages - 1; ph ^= 1u; }
            ok = ptx::mbar_wait(full(s), ph) && ok;
        }
    } else {
        // ------------------------------------------------ products
        const int rw = warp % RW, kw = warp / RW, k0 = kw * NK;
        const int r0 = 16 * rw + lane / 4, r1 = r0 + 8;   // this thread's two rows
        const int tok0 = it.t0 + (it.row0 + r0) / a.group, tok1 = it.t0 + (it.row0 + r1) / a.group;
        const int hq0 = head * a.group + (it.row0 + r0) % a.group, hq1 = head * a.group + (it.row0 + r1) % a.group;
        const bool in0 = r0 < it.rows, in1 = r1 < it.rows;
        uint32_t qf[D / 16][4];
        {
            const uint32_t* q0 = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + tok0 * a.ldq + (long long)hq0 * D) + lane % 4;
            const uint32_t* q1 = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + tok1 * a.ldq + (long long)hq1 * D) + lane % 4;
#pragma unroll
            for (int i = 0; i < D / 16; i++) {
                qf[i][0] = in0 ? __ldg(q0 + 8 * i) : 0u;
                qf[i][1] = in1 ? __ldg(q1 + 8 * i) : 0u;
                qf[i][2] = in0 ? __ldg(q0 + 8 * i + 4) : 0u;
                qf[i][3] = in1 ? __ldg(q1 + 8 * i + 4) : 0u;
            }
        }
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        // shared-memory offsets of the ldmatrix lanes' rows, for each 16 keys; halves of the head are `half` apart
        const uint32_t half = (uint32_t)a.box_rows * 128;
        uint32_t koff[NK / 16], voff[NK / 16];
        const int krow = (lane / 16) * 8 + lane % 8, kchunk = (lane / 8) % 2;
        const int vrow = ((lane / 8) % 2) * 8 + lane % 8, vchunk = lane / 16;
#pragma unroll
        for (int n = 0; n < NK / 16; n++) {
            const int box = (k0 + 16 * n) / a.box_rows, in = (k0 + 16 * n) % a.box_rows;   // 16 keys lie in one box
            koff[n] = box * (half * HALVES) + (in + krow) * 128;
            voff[n] = C::TILE + box * (half * HALVES) + (in + vrow) * 128;
        }

        int s = 0;
        uint32_t ph = 0;
        for (int j = it.tile0; j < it.tile1; j++) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(full(s), ph));
            if (!ok) break;
            const uint32_t kt = sbase + s * C::STAGE;
            // keys k0 .. k0 + vis - 1 of the tile are seen by the row
            const int any = tile_keys(j) - k0;   // ... by any row
            int vis0 = any, vis1 = any;
            if (j >= it.np) {
                const int base = (j - it.np) * KT + k0;
                vis0 = it.own0 + (tok0 - it.t0) - base;
                vis1 = it.own0 + (tok1 - it.t0) - base;
            }
            if (any > 0) {
                if (any < NK) {
                    // V rows past the last key: whatever the page or an older tile left there times a
                    // probability of 0 must be 0 (the row warps of a stage write the same zeros)
                    for (int i = lane; i < (NK - any) * HALVES * 8; i += 32) {
                        const int row = k0 + any + i / (HALVES * 8), c = i % (HALVES * 8);
                        const uint32_t off = s * C::STAGE + C::TILE + (row / a.box_rows) * (half * HALVES) + (c / 8) * half +
                                             (row % a.box_rows) * 128 + (c % 8) * 16;
                        *reinterpret_cast<uint4*>(smem + off) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async();   // the slot's next TMA write comes after these
                    __syncwarp();
                }
                float sc[NK / 8][4];
#pragma unroll
                for (int n = 0; n < NK / 8; n++) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
#pragma unroll
                    for (int n = 0; n < NK / 16; n++) {
                        uint32_t kf[4];
                        ldsm4(kf, kt + koff[n] + (i / 4) * half + ((((2 * i + kchunk) % 8) ^ (lane & 7)) << 4));
                        mma16816<T>(sc[2 * n], qf[i], kf[0], kf[1]);
                        mma16816<T>(sc[2 * n + 1], qf[i], kf[2], kf[3]);
                    }
                }
                if (!__all_sync(0xffffffffu, vis0 >= NK && vis1 >= NK)) {
#pragma unroll
                    for (int n = 0; n < NK / 8; n++) {
                        const int c = 8 * n + 2 * (lane % 4);
                        if (c >= vis0) sc[n][0] = -INFINITY;
                        if (c + 1 >= vis0) sc[n][1] = -INFINITY;
                        if (c >= vis1) sc[n][2] = -INFINITY;
                        if (c + 1 >= vis1) sc[n][3] = -INFINITY;
                    }
                }
                float t0 = sc[0][0], t1 = sc[0][2];
#pragma unroll
                for (int n = 0; n < NK / 8; n++) {
                    t0 = fmaxf(t0, fmaxf(sc[n][0], sc[n][1]));
                    t1 = fmaxf(t1, fmaxf(sc[n][2], sc[n][3]));
                }
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
                const float n0 = fmaxf(m0, t0 * a.scale_log2), n1 = fmaxf(m1, t1 * a.scale_log2);
                // a row that has seen nothing yet has m = -inf: subtract 0 instead (all its terms are 2^-inf)
                const float u0 = n0 == -INFINITY ? 0.0f : n0, u1 = n1 == -INFINITY ? 0.0f : n1;
                if (!__all_sync(0xffffffffu, n0 == m0 && n1 == m1)) {
                    const float f0 = exp2_approx(m0 - u0), f1 = exp2_approx(m1 - u1);
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        o[i][0] *= f0; o[i][1] *= f0;
                        o[i][2] *= f1; o[i][3] *= f1;
                    }
                    m0 = n0;
                    m1 = n1;
                }
                uint32_t pf[NK / 16][4];
#pragma unroll
                for (int n = 0; n < NK / 8; n++) {
                    const float p0 = exp2_approx(fmaf(sc[n][0], a.scale_log2, -u0));
                    const float p1 = exp2_approx(fmaf(sc[n][1], a.scale_log2, -u0));
                    const float p2 = exp2_approx(fmaf(sc[n][2], a.scale_log2, -u1));
                    const float p3 = exp2_approx(fmaf(sc[n][3], a.scale_log2, -u1));
                    l0 += p0 + p1;
                    l1 += p2 + p3;
                    pf[n / 2][2 * (n % 2)] = kv::pack2<T>(p0, p1);
                    pf[n / 2][2 * (n % 2) + 1] = kv::pack2<T>(p2, p3);
                }
#pragma unroll
                for (int n = 0; n < NK / 16; n++) {
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        uint32_t vf[4];
                        ldsm4t(vf, kt + voff[n] + (i / 4) * half + ((((2 * i + vchunk) % 8) ^ (lane & 7)) << 4));
                        mma16816<T>(o[2 * i], pf[n], vf[0], vf[1]);
                        mma16816<T>(o[2 * i + 1], pf[n], vf[2], vf[3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty(s));
            if (++s == stages) { s = 0; ph ^= 1u; }
        }
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);

        // ------------------------------------------------ join the key ranges: the upper half of the warps into the lower
        float4* slots = reinterpret_cast<float4*>(smem);
        float2* mls = reinterpret_cast<float2*>(smem + stages * C::STAGE + C::OFF_ML);
#pragma unroll
        for (int step = KW / 2; step > 0; step /= 2) {
            consumer_sync();   // the stages, or the last step's slots, are no longer read
            if (kw >= step && kw < 2 * step) {
                const int slot = (kw - step) * RW + rw;
#pragma unroll
                for (int i = 0; i < D / 8; i++)
                    slots[(slot * (D / 8) + i) * 32 + lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                if (lane % 4 == 0) {
                    mls[slot * 16 + lane / 4] = make_float2(m0, l0);
                    mls[slot * 16 + lane / 4 + 8] = make_float2(m1, l1);
                }
            }
            consumer_sync();
            if (kw < step) {
                const int slot = kw * RW + rw;
                const float2 p0 = mls[slot * 16 + lane / 4], p1 = mls[slot * 16 + lane / 4 + 8];
                const float n0 = fmaxf(m0, p0.x), n1 = fmaxf(m1, p1.x);
                const float u0 = n0 == -INFINITY ? 0.0f : n0, u1 = n1 == -INFINITY ? 0.0f : n1;
                const float f0 = exp2_approx(m0 - u0), f1 = exp2_approx(m1 - u1);
                const float g0 = exp2_approx(p0.x - u0), g1 = exp2_approx(p1.x - u1);
                l0 = l0 * f0 + p0.y * g0;
                l1 = l1 * f1 + p1.y * g1;
                m0 = n0;
                m1 = n1;
#pragma unroll
                for (int i = 0; i < D / 8; i++) {
                    const float4 v = slots[(slot * (D / 8) + i) * 32 + lane];
                    o[i][0] = o[i][0] * f0 + v.x * g0;
                    o[i][1] = o[i][1] * f0 + v.y * g0;
                    o[i][2] = o[i][2] * f1 + v.z * g1;
                    o[i][3] = o[i][3] * f1 + v.w * g1;
                }
            }
        }
        if (kw == 0) {
            const bool final = a.part_o == nullptr;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                if (!(e ? in1 : in0)) continue;
                const int tok = e ? tok1 : tok0, hq = e ? hq1 : hq0;
                const float m = e ? m1 : m0, l = e ? l1 : l0;
                const long long row = (long long)tok * a.heads_q + hq;
                if (final) {
                    const float inv = inverse(l);
#pragma unroll
                    for (int i = 0; i < D / 8; i++)
                        store_out2(a, tok * a.ldo + (long long)hq * D + 8 * i + 2 * (lane % 4), o[i][2 * e] * inv,
                                   o[i][2 * e + 1] * inv);
                    if (lane % 4 == 0) store_lse(a, row, m, l);
                } else {
                    const long long at = (long long)(sp.part0 + part) * a.rows + row;
                    if (lane % 4 == 0) a.part_ml[at] = make_float2(m, l);
                    if (l != 0.0f)
#pragma unroll
                        for (int i = 0; i < D / 8; i++)
                            *reinterpret_cast<float2*>(a.part_o + at * D + 8 * i + 2 * (lane % 4)) =
                                make_float2(o[i][2 * e], o[i][2 * e + 1]);
                }
            }
        }
    }
    if (!ok && a.status) atomicExch(a.status, (int)QG_ERR_TIMEOUT);
}

template <typename T, int D, int RW, int KEYS>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3)
    k_attn_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ Args a, const __grid_constant__ Split sp, int stages, int beside)
{
    work<T, D, RW, KEYS>(kmap, vmap, a, sp, blockIdx.x, stages, beside != 0);
}

// The shared prefix for all rows (its CTAs first) and the own tokens in one launch.
template <typename T, int D, int RWP, int RWO>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3)
    k_attn_rows_shared(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ Args a, const __grid_constant__ Split prefix,
                       const __grid_constant__ Split own, int prefix_ctas, int stages)
{
    if ((int)blockIdx.x < prefix_ctas) work<T, D, RWP, kPrefix>(kmap, vmap, a, prefix, blockIdx.x, stages, false);
    else work<T, D, RWO, kOwn>(kmap, vmap, a, own, (int)blockIdx.x - prefix_ctas, stages, false);
}

// Row blocks of 16 rows that a CTA takes for so many rows a unit.
int row_warps(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

struct Launch {
    Split sp;
    int64_t ctas;
};
Launch plan(const Args& a, int keys, int rw, int part0, int parts, int most_tiles, bool beside = false)
{
    const int64_t units = (keys & kOwn) ? a.bt.B : 1;
    const int64_t blocks = ceil_div((int64_t)a.group * ((keys & kOwn) ? a.bt.max_q : a.bt.T), 16 * rw);
    const int least = std::min(beside ? kLeastBeside : kLeastTiles, most_tiles);
    return Launch{Split{part0, parts, least, (int)blocks}, units * blocks * parts * a.c.heads};
}

// No more stages than tiles: more of the shared memory stays with the kernel beside.
template <int D> int stages_for(int tiles) { return std::max(1, std::min(tiles, Cfg<D>::MAX_STAGES)); }
template <int D> int smem_for(int stages) { return stages * Cfg<D>::STAGE + Cfg<D>::REST; }

template <typename T, int D, int RW, int KEYS>
cudaError_t launch_one(const Args& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int part0, int parts,
                       int most_tiles, bool beside, cudaStream_t s)
{
    auto kernel = k_attn_rows<T, D, RW, KEYS>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = kv::allow_smem(kernel, smem_for<D>(Cfg<D>::MAX_STAGES), done);
    if (e != cudaSuccess) return e;
    const Launch l = plan(a, KEYS, RW, part0, parts, most_tiles, beside);
    if (l.ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int stages = stages_for<D>(most_tiles);
    return kv::launch_dependent(kernel, dim3((unsigned)l.ctas), kThreads, smem_for<D>(stages), s, kmap, vmap, a, l.sp,
                                stages, beside ? 1 : 0);
}

template <typename T, int D, int RWP, int RWO>
cudaError_t launch_both(const Args& a, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& p, cudaStream_t s)
{
    auto kernel = k_attn_rows_shared<T, D, RWP, RWO>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = kv::allow_smem(kernel, smem_for<D>(Cfg<D>::MAX_STAGES), done);
    if (e != cudaSuccess) return e;
    const Launch l = plan(a, kPrefix, RWP, 0, p.prefix_parts, p.prefix_tiles);
    const Launch m = plan(a, kOwn, RWO, p.prefix_parts, p.own_parts, p.own_tiles);
    if (l.ctas + m.ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int stages = stages_for<D>(std::max(p.prefix_tiles, p.own_tiles));
    return kv::launch_dependent(kernel, dim3((unsigned)(l.ctas + m.ctas)), kThreads, smem_for<D>(stages), s, kmap, vmap, a,
                                l.sp, m.sp, (int)l.ctas, stages);
}

template <typename T, int D>
cudaError_t by_keys(const Args& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int keys, const Parts& p, bool beside,
                    cudaStream_t s)
{
    const int part0 = keys == kOwn ? p.prefix_parts : 0, n = p.own_parts, t = p.own_tiles;
    const int rw = row_warps((int64_t)a.group * a.bt.max_q);
    if (keys == kOwn)
        return rw == 1   ? launch_one<T, D, 1, kOwn>(a, kmap, vmap, part0, n, t, beside, s)
               : rw == 2 ? launch_one<T, D, 2, kOwn>(a, kmap, vmap, part0, n, t, beside, s)
                         : launch_one<T, D, 4, kOwn>(a, kmap, vmap, part0, n, t, beside, s);
    return rw == 1   ? launch_one<T, D, 1, kPrefix | kOwn>(a, kmap, vmap, part0, n, t, beside, s)
           : rw == 2 ? launch_one<T, D, 2, kPrefix | kOwn>(a, kmap, vmap, part0, n, t, beside, s)
                     : launch_one<T, D, 4, kPrefix | kOwn>(a, kmap, vmap, part0, n, t, beside, s);
}

template <typename T, int D>
cudaError_t both(const Args& a, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& p, cudaStream_t s)
{
    const int rw = row_warps((int64_t)a.group * a.bt.max_q);
    if ((int64_t)a.group * a.bt.T <= 16) return launch_both<T, D, 1, 1>(a, kmap, vmap, p, s);
    return rw == 1   ? launch_both<T, D, 4, 1>(a, kmap, vmap, p, s)
           : rw == 2 ? launch_both<T, D, 4, 2>(a, kmap, vmap, p, s)
                     : launch_both<T, D, 4, 4>(a, kmap, vmap, p, s);
}

}  // namespace

cudaError_t launch_rows(const Args& a, int dtype, const CUtensorMap& kmap, const CUtensorMap& vmap, int keys,
                        const Parts& p, bool beside, cudaStream_t s)
{
    if (dtype == QG_T_BF16)
        return a.c.dim == 128 ? by_keys<__nv_bfloat16, 128>(a, kmap, vmap, keys, p, beside, s)
                              : by_keys<__nv_bfloat16, 64>(a, kmap, vmap, keys, p, beside, s);
    return a.c.dim == 128 ? by_keys<__half, 128>(a, kmap, vmap, keys, p, beside, s)
                          : by_keys<__half, 64>(a, kmap, vmap, keys, p, beside, s);
}

cudaError_t launch_rows_shared(const Args& a, int dtype, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& p,
                               cudaStream_t s)
{
    if (dtype == QG_T_BF16)
        return a.c.dim == 128 ? both<__nv_bfloat16, 128>(a, kmap, vmap, p, s) : both<__nv_bfloat16, 64>(a, kmap, vmap, p, s);
    return a.c.dim == 128 ? both<__half, 128>(a, kmap, vmap, p, s) : both<__half, 64>(a, kmap, vmap, p, s);
}

}  // namespace attn
}  // namespace qg
