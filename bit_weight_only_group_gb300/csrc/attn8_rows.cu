// Attention over the 8-bit cache for few query rows per key/value head: the row
// kernel of attn_rows.cu with codes in place of 16-bit values.
//
// K and V codes stream through shared memory by TMA, half the bytes a key, and
// become fp16 between shared memory and the products, two codes an instruction
// (measured 59 such conversions a clock and SM; the keys that HBM delivers need
// 12).  ldmatrix moves pairs of bytes, so
//  K: a thread gets four neighbouring codes of a key, which serve as the two
//     pairs of a step's 16 values of the head in another order, the same that
//     q's registers have;
//  V: transposed, a thread gets two keys' codes of two neighbouring columns, a
//     byte permutation puts each column's two keys together, and the columns of
//     a pair go to two products: a thread ends up with four neighbouring ones.
// Scales and their use: attn.cuh.  The loading warp looks up pages and scale
// bytes, a chain of two loads, for 256 keys at a time (a lane for the K or the V
// of 16), one and two such batches ahead of the copies it issues, and leaves 2^e
// beside the stage.
#include "attn_rows.cuh"

namespace qg {
namespace attn {
namespace {

// Keys of a stage: with one row block the four warps share them, 32 each; with four every warp takes all.
template <int RW> constexpr int kKeys = RW == 4 ? 64 : 128;

template <int D, int RW> struct Cfg8 {
    static constexpr int KT = kKeys<RW>, GROUPS = KT / kv8::kBlock;
    static constexpr int MAX_STAGES = KT == 128 ? (D == 128 ? 3 : 5) : (D == 128 ? 6 : 8);
    static constexpr int TILE = KT * D;                  // bytes of a K or V tile: [key][dim], swizzled
    static constexpr int STAGE = 2 * TILE;
    static constexpr int SCALES = 3 * GROUPS;            // floats of a stage: 2^ek scale log2(e), ev, 2^-ev
    static constexpr int OFF_SCALES = 2 * 8 * MAX_STAGES;   // after the barriers
    static constexpr int OFF_ML = OFF_SCALES + MAX_STAGES * SCALES * 4;
    static constexpr int REST = OFF_ML + kWarps * 16 * 8 + 1024;   // barriers, scales, (m, l), alignment
    static_assert(2 * 16 * D * 4 <= STAGE, "joining buffers fit a stage");
    // offset of a 16-byte chunk of a row: the swizzle of 128-byte, or of 64-byte, boxes
    static __device__ __forceinline__ uint32_t at(int row, int chunk)
    {
        return (uint32_t)(row * D + ((chunk ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4));
    }
};

template <int D, int RW, int KEYS>
__device__ __forceinline__ void work8(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args8& p8, const Split& sp,
                                      int x, int stages, bool beside)
{
    using C = Cfg8<D, RW>;
    constexpr int KT = C::KT, GROUPS = C::GROUPS, KW = kWarps / RW, NK = KT / KW, NG = NK / 16;
    const Args& a = p8.a;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem), bars = sbase + stages * C::STAGE;
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (C::MAX_STAGES + s); };
    float* scales = reinterpret_cast<float*>(smem + stages * C::STAGE + C::OFF_SCALES);
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
    const Item it = find_item<KEYS, KT>(a, unit, row_block, part, sp.parts, sp.least_tiles, 16 * RW, threadIdx.x == 0);
    if (it.rows == 0) return;
    bool ok = true;
    // keys of tile j that any row sees
    auto tile_keys = [&](int j) { return j < it.np ? min(KT, it.prefix - j * KT) : min(KT, it.own - (j - it.np) * KT); };

    if (warp == kWarps) {
        // ------------------------------------------------ loads: a lane each for the K or the V of 16 keys
        constexpr int LANES = 2 * GROUPS, BATCH = 32 / LANES;   // of a tile; tiles of a batch
        const int turn = lane / LANES, group = lane % GROUPS, is_v = lane % LANES / GROUPS;
        const bool boxes = group * 16 % a.box_rows == 0;        // the first lane of a page's rows loads them
        const int* own_table = (KEYS & kOwn) ? a.bt.table + (long long)it.b * a.bt.table_ld : nullptr;
        const int mask = (1 << a.c.page_shift) - 1;
        auto key_of = [&](int j) { return (j < it.np ? j : j - it.np) * KT + group * 16; };
        auto entry_at = [&](int j) {   // of the table, for this lane's keys of tile j
            const bool there = j < it.tile1 && group * 16 < tile_keys(j);
            return table_entry(a, j < it.np ? a.bt.prefix_table : own_table, key_of(j) >> a.c.page_shift, there);
        };
        auto byte_at = [&](int page, int j) { return scale_byte(p8, is_v != 0, page, (key_of(j) & mask) / 16, head); };
        int s = 0, issued = 0;
        uint32_t ph = 0;
        int mine = it.tile0 + turn;   // this lane's tile of the batch
        int page = checked_page(a, entry_at(mine)), byte = byte_at(page, mine);
        Entry next = entry_at(mine + BATCH);
        for (int j0 = it.tile0; ok && j0 < it.tile1; j0 += BATCH, mine += BATCH) {
            const int next_page = checked_page(a, next), next_byte = byte_at(next_page, mine + BATCH);
            const int e = scale_exp(byte);
            next = entry_at(mine + 2 * BATCH);
            for (int t = 0; t < BATCH && j0 + t < it.tile1; t++) {
                const int j = j0 + t;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(empty(s), ph ^ 1u));
                if (!ok) break;
                if (turn == t) {
                    float* to = scales + s * C::SCALES + group;
                    if (!is_v) {
                        to[0] = a.scale_log2 * kv8::pow2(e);
                    } else {
                        to[GROUPS] = (float)e;
                        to[2 * GROUPS] = kv8::pow2(-e);
                    }
                }
                __syncwarp();
                const int used = (tile_keys(j) + a.box_rows - 1) / a.box_rows;
                if (lane == 0) ptx::mbar_expect_tx(full(s), (uint32_t)(used * a.box_rows * (2 * D)));
                __syncwarp();
                if (turn == t && boxes && group * 16 < used * a.box_rows)
                    tma_load_4d(sbase + s * C::STAGE + is_v * C::TILE + group * 16 * D, is_v ? &vmap : &kmap, 0,
                                key_of(j) & mask, head, page, full(s));
                issued++;
                if (++s == stages) { s = 0; ph ^= 1u; }
            }
            page = next_page;
            byte = next_byte;
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
        float back0, back1;   // 2^(x - 14): what the rows' q was scaled by, undone on the logits
        {
            const uint2* q0 = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + tok0 * a.ldq + (long long)hq0 * D) + lane % 4;
            const uint2* q1 = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + tok1 * a.ldq + (long long)hq1 * D) + lane % 4;
            uint2 w[2][D / 16];
#pragma unroll
            for (int i = 0; i < D / 16; i++) {
                w[0][i] = in0 ? __ldg(q0 + 4 * i) : make_uint2(0u, 0u);
                w[1][i] = in1 ? __ldg(q1 + 4 * i) : make_uint2(0u, 0u);
            }
            const bool bf = p8.q_type == QG_T_BF16;
            auto value = [&](uint32_t u) {
                return bf ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u)) : kv8::half2_floats(u);
            };
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
                    const float2 u = value(w[e][i].x), v = value(w[e][i].y);
                    amax = fmaxf(fmaxf(fmaxf(amax, fabsf(u.x)), fabsf(u.y)), fmaxf(fabsf(v.x), fabsf(v.y)));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const int ex = row_exp(amax);
                const float up = kv8::pow2(min(14 - ex, 127));
                (e ? back1 : back0) = kv8::pow2(ex - 14);
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
                    const float2 u = value(w[e][i].x), v = value(w[e][i].y);
                    qf[i][e] = kv::pack2<__half>(u.x * up, u.y * up);
                    qf[i][2 + e] = kv::pack2<__half>(v.x * up, v.y * up);
                }
            }
        }
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        // the ldmatrix lanes' rows and chunks
        const int krow = (lane / 16) * 8 + lane % 8, kchunk = (lane / 8) % 2;
        const int vrow = ((lane / 8) % 2) * 8 + lane % 8, vchunk = lane / 16;

        int s = 0;
        uint32_t ph = 0;
        for (int j = it.tile0; j < it.tile1; j++) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(full(s), ph));
            if (!ok) break;
            const uint32_t kt = sbase + s * C::STAGE, vt = kt + C::TILE;
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
                    for (int i = lane; i < (NK - any) * (D / 16); i += 32)
                        *reinterpret_cast<uint4*>(smem + s * C::STAGE + C::TILE + (k0 + any + i / (D / 16)) * D + i % (D / 16) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    ptx::fence_proxy_async();   // the slot's next TMA write comes after these
                    __syncwarp();
                }
                float sc[NK / 8][4];
#pragma unroll
                for (int n = 0; n < NK / 8; n++) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; i += 2) {
#pragma unroll
                    for (int n = 0; n < NG; n++) {
                        uint32_t kf[4];   // keys 0-7 of chunks i and i + 1, keys 8-15 of the same
                        ldsm4(kf, kt + C::at(k0 + 16 * n + krow, i + kchunk));
                        mma16816<__half>(sc[2 * n], qf[i], kv8::decode_lo(kf[0]), kv8::decode_hi(kf[0]));
                        mma16816<__half>(sc[2 * n + 1], qf[i], kv8::decode_lo(kf[2]), kv8::decode_hi(kf[2]));
                        mma16816<__half>(sc[2 * n], qf[i + 1], kv8::decode_lo(kf[1]), kv8::decode_hi(kf[1]));
                        mma16816<__half>(sc[2 * n + 1], qf[i + 1], kv8::decode_lo(kf[3]), kv8::decode_hi(kf[3]));
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
                // s + ev of a group: the raw logits times f, plus ev (f at least the smallest normal number: a masked
                // logit times 0 would be a NaN)
                const float* stage = scales + s * C::SCALES + k0 / 16;
                float f0[NG], f1[NG], ev[NG], t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int n = 0; n < NG; n++) {
                    const float k = stage[n];
                    ev[n] = stage[GROUPS + n];
                    f0[n] = fmaxf(k * back0, 1.17549435e-38f);
                    f1[n] = fmaxf(k * back1, 1.17549435e-38f);
                    t0 = fmaxf(t0, fmaf(fmaxf(fmaxf(sc[2 * n][0], sc[2 * n][1]), fmaxf(sc[2 * n + 1][0], sc[2 * n + 1][1])), f0[n], ev[n]));
                    t1 = fmaxf(t1, fmaf(fmaxf(fmaxf(sc[2 * n][2], sc[2 * n][3]), fmaxf(sc[2 * n + 1][2], sc[2 * n + 1][3])), f1[n], ev[n]));
                }
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
                const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
                // a row that has seen nothing yet has m = -inf: subtract 0 instead (all its terms are 2^-inf)
                const float u0 = n0 == -INFINITY ? 0.0f : n0, u1 = n1 == -INFINITY ? 0.0f : n1;
                if (!__all_sync(0xffffffffu, n0 == m0 && n1 == m1)) {
                    const float g0 = exp2_approx(m0 - u0), g1 = exp2_approx(m1 - u1);
                    l0 *= g0;
                    l1 *= g1;
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        o[i][0] *= g0; o[i][1] *= g0;
                        o[i][2] *= g1; o[i][3] *= g1;
                    }
                    m0 = n0;
                    m1 = n1;
                }
                uint32_t pf[NG][4];
#pragma unroll
                for (int n = 0; n < NG; n++) {
                    float p[8];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        p[2 * e] = exp2_approx(fmaf(sc[2 * n + e / 2][2 * (e % 2)], e % 2 ? f1[n] : f0[n], ev[n] - (e % 2 ? u1 : u0)));
                        p[2 * e + 1] = exp2_approx(fmaf(sc[2 * n + e / 2][2 * (e % 2) + 1], e % 2 ? f1[n] : f0[n], ev[n] - (e % 2 ? u1 : u0)));
                        pf[n][e] = kv::pack2<__half>(p[2 * e], p[2 * e + 1]);
                    }
                    const float iv = stage[2 * GROUPS + n];
                    l0 = fmaf((p[0] + p[1]) + (p[4] + p[5]), iv, l0);
                    l1 = fmaf((p[2] + p[3]) + (p[6] + p[7]), iv, l1);
                }
#pragma unroll
                for (int n = 0; n < NG; n++) {
#pragma unroll
                    for (int i = 0; i < D / 16; i += 2) {
                        uint32_t vf[4];   // keys 0-7 and 8-15 of chunk i, of chunk i + 1
                        ldsm4t(vf, vt + C::at(k0 + 16 * n + vrow, i + vchunk));
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const uint32_t lo = __byte_perm(vf[2 * h], 0u, 0x3120), hi = __byte_perm(vf[2 * h + 1], 0u, 0x3120);
                            mma16816<__half>(o[2 * (i + h)], pf[n], kv8::decode_lo(lo), kv8::decode_lo(hi));
                            mma16816<__half>(o[2 * (i + h) + 1], pf[n], kv8::decode_hi(lo), kv8::decode_hi(hi));
                        }
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
                // the thread's four neighbouring columns of chunk i lie in the two products of the chunk in turn
                auto four = [&](int i, float w) {
                    return make_float4(o[2 * i][2 * e] * w, o[2 * i + 1][2 * e] * w, o[2 * i][2 * e + 1] * w, o[2 * i + 1][2 * e + 1] * w);
                };
                if (final) {
                    const float inv = inverse(l);
#pragma unroll
                    for (int i = 0; i < D / 16; i++) store_out4(a, tok * a.ldo + (long long)hq * D + 16 * i + 4 * (lane % 4), four(i, inv));
                    if (lane % 4 == 0) store_lse(a, row, m, l);
                } else {
                    const long long at = (long long)(sp.part0 + part) * a.rows + row;
                    if (lane % 4 == 0) a.part_ml[at] = make_float2(m, l);
                    if (l != 0.0f)
#pragma unroll
                        for (int i = 0; i < D / 16; i++)
                            *reinterpret_cast<float4*>(a.part_o + at * D + 16 * i + 4 * (lane % 4)) = four(i, 1.0f);
                }
            }
        }
    }
    if (!ok && a.status) atomicExch(a.status, (int)QG_ERR_TIMEOUT);
}

template <int D, int RW, int KEYS>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3)
    k_attn8_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ Args8 p, const __grid_constant__ Split sp, int stages, int beside)
{
    work8<D, RW, KEYS>(kmap, vmap, p, sp, blockIdx.x, stages, beside != 0);
}

// The shared prefix for all rows (its CTAs first) and the own tokens in one launch.
template <int D, int RWP, int RWO>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3)
    k_attn8_rows_shared(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ Args8 p, const __grid_constant__ Split prefix,
                        const __grid_constant__ Split own, int prefix_ctas, int prefix_stages, int own_stages)
{
    if ((int)blockIdx.x < prefix_ctas) work8<D, RWP, kPrefix>(kmap, vmap, p, prefix, blockIdx.x, prefix_stages, false);
    else work8<D, RWO, kOwn>(kmap, vmap, p, own, (int)blockIdx.x - prefix_ctas, own_stages, false);
}

// Shared memory of a CTA for parts of so many 64-key tiles: no more stages than it has use for, so that more stays with
// the kernel beside.
template <int D, int RW> int stages_for(int tiles)
{
    return std::max(1, std::min((int)ceil_div(tiles, kKeys<RW> / 64), Cfg8<D, RW>::MAX_STAGES));
}
template <int D, int RW> int smem_for(int stages) { return stages * Cfg8<D, RW>::STAGE + Cfg8<D, RW>::REST; }

template <int D, int RW, int KEYS>
cudaError_t launch_one(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int part0, int parts,
                       int most_tiles, bool beside, cudaStream_t s)
{
    auto kernel = k_attn8_rows<D, RW, KEYS>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = kv::allow_smem(kernel, smem_for<D, RW>(Cfg8<D, RW>::MAX_STAGES), done);
    if (e != cudaSuccess) return e;
    const Launch l = plan(p.a, KEYS, RW, part0, parts, most_tiles, beside, kKeys<RW>);
    if (l.ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int stages = stages_for<D, RW>(most_tiles);
    return kv::launch_dependent(kernel, dim3((unsigned)l.ctas), kThreads, smem_for<D, RW>(stages), s, kmap, vmap, p, l.sp,
                                stages, beside ? 1 : 0);
}

template <int D, int RWP, int RWO>
cudaError_t launch_both(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& n, cudaStream_t s)
{
    auto kernel = k_attn8_rows_shared<D, RWP, RWO>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = kv::allow_smem(kernel, std::max(smem_for<D, RWP>(Cfg8<D, RWP>::MAX_STAGES),
                                                          smem_for<D, RWO>(Cfg8<D, RWO>::MAX_STAGES)), done);
    if (e != cudaSuccess) return e;
    const Launch l = plan(p.a, kPrefix, RWP, 0, n.prefix_parts, n.prefix_tiles, false, kKeys<RWP>);
    const Launch m = plan(p.a, kOwn, RWO, n.prefix_parts, n.own_parts, n.own_tiles, false, kKeys<RWO>);
    if (l.ctas + m.ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int ps = stages_for<D, RWP>(n.prefix_tiles), os = stages_for<D, RWO>(n.own_tiles);
    const int smem = std::max(smem_for<D, RWP>(ps), smem_for<D, RWO>(os));
    return kv::launch_dependent(kernel, dim3((unsigned)(l.ctas + m.ctas)), kThreads, smem, s, kmap, vmap, p, l.sp, m.sp,
                                (int)l.ctas, ps, os);
}

template <int D>
cudaError_t by_keys(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int keys, const Parts& n, bool beside,
                    cudaStream_t s)
{
    const int part0 = keys == kOwn ? n.prefix_parts : 0, parts = n.own_parts, t = n.own_tiles;
    const int rw = row_warps((int64_t)p.a.group * p.a.bt.max_q);
    if (keys == kOwn)
        return rw == 1   ? launch_one<D, 1, kOwn>(p, kmap, vmap, part0, parts, t, beside, s)
               : rw == 2 ? launch_one<D, 2, kOwn>(p, kmap, vmap, part0, parts, t, beside, s)
                         : launch_one<D, 4, kOwn>(p, kmap, vmap, part0, parts, t, beside, s);
    return rw == 1   ? launch_one<D, 1, kPrefix | kOwn>(p, kmap, vmap, part0, parts, t, beside, s)
           : rw == 2 ? launch_one<D, 2, kPrefix | kOwn>(p, kmap, vmap, part0, parts, t, beside, s)
                     : launch_one<D, 4, kPrefix | kOwn>(p, kmap, vmap, part0, parts, t, beside, s);
}

template <int D>
cudaError_t both(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& n, cudaStream_t s)
{
    const int rw = row_warps((int64_t)p.a.group * p.a.bt.max_q);
    if ((int64_t)p.a.group * p.a.bt.T <= 16) return launch_both<D, 1, 1>(p, kmap, vmap, n, s);
    return rw == 1   ? launch_both<D, 4, 1>(p, kmap, vmap, n, s)
           : rw == 2 ? launch_both<D, 4, 2>(p, kmap, vmap, n, s)
                     : launch_both<D, 4, 4>(p, kmap, vmap, n, s);
}

}  // namespace

cudaError_t launch_rows8(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int keys, const Parts& n,
                         bool beside, cudaStream_t s)
{
    return p.a.c.dim == 128 ? by_keys<128>(p, kmap, vmap, keys, n, beside, s) : by_keys<64>(p, kmap, vmap, keys, n, beside, s);
}

cudaError_t launch_rows8_shared(const Args8& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const Parts& n,
                                cudaStream_t s)
{
    return p.a.c.dim == 128 ? both<128>(p, kmap, vmap, n, s) : both<64>(p, kmap, vmap, n, s);
}

}  // namespace attn
}  // namespace qg
