// Appending to the 8-bit paged cache, and reading it back.
//
// Keys (normed and turned) and values become E4M3 codes with one power of two
// for 16 places of a page and head: with amax the largest magnitude among a
// block's new values, e is the least integer with amax <= 448 * 2^e and a code
// the nearest E4M3 value of x 2^-e.  A power of two loses E4M3 nothing (its
// precision is relative), needs no division, and lets the scale of a block that
// later tokens grow be raised with its codes rounded again only where they
// become subnormal.
//
// Bound by HBM: a value is read once and written once.  A unit of work is the
// new tokens of one sequence in one block of places; a CTA takes a unit and
// some heads, a warp one head at a time with all (up to 16) tokens in
// registers, so that the largest magnitude needs shuffles alone and nothing is
// read twice.  The unit's cosines and sines are staged in shared memory, once
// for all heads.  With one new token a sequence the rows of a warp are heads.
// Appending and reading back: one token into 40 8.2 us, 256 into sequences of up
// to 512 (16 heads of 128 read back, 416 MB in all) 84.9 us, 4.9 TB/s; prompts of
// 4200 tokens of 32 + 2 x 8 heads of 64 28.6 us (72 MB), two launches whose CTAs
// wait for offsets, lengths, table and data one after another.
#include <algorithm>

#include "kv8.cuh"
#include "kv_heads.cuh"

namespace qg {
namespace kv8 {
namespace {

struct AppendArgs {
    kv::Batch bt;
    Cache c;
    uint8_t *kc, *vc, *ks, *vs;
    const void *q, *k, *v;
    long long ldq, ldk, ldv, ldq_out;
    void* q_out;
    int qt, heads_q;
    const float* rope;   // null: no rotation
    const int* at;
    int positions, rot, interleaved;
    kv::Norm norm;
    int* status;
};

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeadsEach = 2;   // heads a warp takes one after another, at most

// Place of a unit in a page, and of its scale.
__device__ __forceinline__ long long codes_at(const Cache& c, const Unit& x, int slot, int head)
{
    const int in_page = (x.block * kBlock & ((1 << c.page_shift) - 1)) + slot;
    return (long long)x.page * c.page_stride + (long long)in_page * c.token_stride + (long long)head * c.head_stride;
}
__device__ __forceinline__ long long scale_at(const Cache& c, const Unit& x, int head)
{
    const int in_page = (x.block * kBlock & ((1 << c.page_shift) - 1)) >> kBlockShift;
    return (long long)x.page * c.scale_page + (long long)in_page * c.scale_block + (long long)head * c.scale_head;
}

// SINGLE: at most one new token a sequence; a warp's rows are then heads, else places of the block.
template <typename TI, int D, bool SINGLE>
__global__ void __launch_bounds__(kThreads, D == 64 ? 3 : 2) k_kv8_append(const __grid_constant__ AppendArgs a)
{
    constexpr int LANES = D / 16, ROWS = 32 / LANES, ITER = SINGLE ? 1 : kBlock / ROWS;
    constexpr int HEADS = SINGLE ? ROWS : 1;                 // heads of a warp at a time
    __shared__ float4 weights[8 * LANES];                    // of the norms (stage_weights)
    __shared__ __align__(16) float angles[SINGLE ? 1 : kBlock][D];
    __shared__ bool live[kBlock];                            // the token's position is in the table
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = lane % LANES, row = lane / LANES;
    kv::pdl_wait();      // the values, lengths and tables may come from the kernel just before
    kv::pdl_release();
    if (blockIdx.y == 0) check_lengths(a.bt, a.status);
    Unit x;
    if (!find_unit(a.bt, a.c, blockIdx.x, x)) return;
    const bool normed = a.norm.q || a.norm.k;
    // where in a turned head a lane's two runs of 8 values are, and in a value head
    const bool turn = a.rope && j < a.rot / 16;
    const int t0 = turn && !a.interleaved ? 8 * j : 16 * j, t1 = turn && !a.interleaved ? a.rot / 2 + 8 * j : 16 * j + 8;
    if (normed) kv::stage_weights<LANES>(weights, a.norm, a.rot, a.interleaved);
    // the row of the rotation table of the token at a place, or -1
    auto position = [&](int slot) -> long long {
        const int t = x.t0 + slot - x.s0;
        const long long p = a.at ? (long long)__ldg(a.at + t) : (long long)a.bt.prefix_len + x.block * kBlock + slot;
        return p >= 0 && p < a.positions ? p : -1;
    };
    if (threadIdx.x < kBlock) {
        const int slot = threadIdx.x;
        bool ok = slot >= x.s0 && slot < x.s1;
        if (ok && a.rope && position(slot) < 0) {
            ok = false;
            if (blockIdx.y == 0) kv::report(a.status);
        }
        live[slot] = ok;
    }
    if (!x.ok && blockIdx.y == 0 && threadIdx.x == 0) kv::report(a.status);
    if (!SINGLE && a.rope) {
        const int per = a.rot / 4;   // float4 of a row
        for (int i = threadIdx.x; i < (x.s1 - x.s0) * per; i += kThreads) {
            const int slot = x.s0 + i / per;
            const long long p = position(slot);
            if (p >= 0) reinterpret_cast<float4*>(angles[slot])[i % per] = __ldg(reinterpret_cast<const float4*>(a.rope + p * a.rot) + i % per);
        }
    }
    __syncthreads();

    const int hq = a.heads_q, hk = a.c.heads, heads = hq + 2 * hk;
    for (int n = 0; n < kHeadsEach; n++) {
        const int first = ((blockIdx.y * kHeadsEach + n) * kWarps + warp) * HEADS;
        if (first >= heads) return;
        const int head = SINGLE ? first + row : first;
        const bool there = head < heads;
        const bool value = head >= hq + hk, key = head >= hq && !value;
        const int i0 = value ? 16 * j : t0, i1 = value ? 16 * j + 8 : t1;
        const TI* src = static_cast<const TI*>(value ? a.v : key ? a.k : a.q);
        const long long ld = value ? a.ldv : key ? a.ldk : a.ldq;
        const int h = value ? head - hq - hk : key ? head - hq : head;
        float f[ITER][2][8];
        bool in[ITER];
        kv::Run8<TI> raw[ITER][2];
#pragma unroll
        for (int i = 0; i < ITER; i++) {
            const int slot = SINGLE ? x.s0 : i * ROWS + row;
            in[i] = there && live[slot];
            if (in[i]) {
                const TI* p = src + (x.t0 + slot - x.s0) * ld + (long long)h * D;
                raw[i][0] = kv::load8(p + i0);
                raw[i][1] = kv::load8(p + i1);
            } else {
                raw[i][0] = raw[i][1] = kv::Run8<TI>{};
            }
        }
#pragma unroll
        for (int i = 0; i < ITER; i++) {
            kv::to_float(raw[i][0], f[i][0]);
            kv::to_float(raw[i][1], f[i][1]);
            // the shuffles of a head's lanes: `value` and the norms are the same for all of them
            if (!value && (key ? a.norm.k : a.norm.q)) kv::norm_head<LANES, D>(f[i][0], f[i][1], weights + key * 4 * LANES + j, a.norm.eps);
            if (turn && !value && in[i]) {
                float cs[8], sn[8];
                const float* at = SINGLE ? a.rope + position(x.s0) * a.rot : angles[i * ROWS + row];
                kv::to_float(kv::load8(at + 8 * j), cs);
                kv::to_float(kv::load8(at + a.rot / 2 + 8 * j), sn);
                kv::turn16(f[i][0], f[i][1], cs, sn, a.interleaved);
            }
        }
        if (!value && !key) {
#pragma unroll
            for (int i = 0; i < ITER; i++) {
                if (!in[i]) continue;
                const int slot = SINGLE ? x.s0 : i * ROWS + row;
                const long long to = (x.t0 + slot - x.s0) * a.ldq_out + (long long)h * D;
                if (a.qt == QG_T_BF16) {
                    kv::store8(static_cast<__nv_bfloat16*>(a.q_out) + to + i0, f[i][0]);
                    kv::store8(static_cast<__nv_bfloat16*>(a.q_out) + to + i1, f[i][1]);
                } else {
                    kv::store8(static_cast<__half*>(a.q_out) + to + i0, f[i][0]);
                    kv::store8(static_cast<__half*>(a.q_out) + to + i1, f[i][1]);
                }
            }
        }
        // from here on for keys and values; in a warp of several heads the others' lanes come along
        const bool keep = there && head >= hq && x.page >= 0;
        if (!SINGLE && !keep) continue;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < ITER; i++)
#pragma unroll
            for (int r = 0; r < 2; r++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const bool fine = fabsf(f[i][r][e]) <= kMost;
                    if (fine) amax = fmaxf(amax, fabsf(f[i][r][e]));
                    else f[i][r][e] = __int_as_float(0x7FC00000);
                }
#pragma unroll
        for (int i = (SINGLE ? LANES : 32) / 2; i > 0; i /= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, i));
        int e = scale_exp(amax);
        uint8_t* codes = value ? a.vc : a.kc;
        uint8_t* scale = (value ? a.vs : a.ks) + (keep ? scale_at(a.c, x, h) : 0);
        if (x.s0 > 0) {   // earlier tokens' codes
            const int old = keep ? min(max((int)*scale - kBias, kMinExp), kMaxExp) : kMaxExp;
            if (old < e) {
                const float down = pow2(old - e);
                auto follow = [&](int slot) {
                    uint4* p = reinterpret_cast<uint4*>(codes + codes_at(a.c, x, slot, h) + 16 * j);
                    const uint4 w = *p;
                    *p = make_uint4(rescale4(w.x, down), rescale4(w.y, down), rescale4(w.z, down), rescale4(w.w, down));
                };
                if constexpr (SINGLE) {
                    for (int slot = 0; slot < x.s0; slot++) follow(slot);
                } else {
                    for (int slot = row; slot < x.s0; slot += ROWS) follow(slot);
                }
            } else {
                e = old;
            }
        }
        __syncwarp();
        if (!keep) continue;
        if (j == 0 && (SINGLE || row == 0)) *scale = (uint8_t)(e + kBias);
        const float up = pow2(-e);
#pragma unroll
        for (int i = 0; i < ITER; i++) {
            if (!in[i]) continue;
            const int slot = SINGLE ? x.s0 : i * ROWS + row;
            uint32_t w[4];
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const float* g = &f[i][r / 2][4 * (r % 2)];
                w[r] = encode2(g[0] * up, g[1] * up) | encode2(g[2] * up, g[3] * up) << 16;
            }
            uint8_t* p = codes + codes_at(a.c, x, slot, h);
            if (i1 == i0 + 8) {
                *reinterpret_cast<uint4*>(p + i0) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                *reinterpret_cast<uint2*>(p + i0) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(p + i1) = make_uint2(w[2], w[3]);
            }
        }
    }
}

struct ReadArgs {
    kv::Batch bt;
    Cache c;
    const uint8_t *kc, *vc, *ks, *vs;
    void *k, *v;
    long long ldk, ldv;
    int* status;
};

template <typename TO, int D>
__global__ void __launch_bounds__(kThreads) k_kv8_read(const __grid_constant__ ReadArgs a)
{
    constexpr int LANES = D / 16, ROWS = 32 / LANES, ITER = kBlock / ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = lane % LANES, row = lane / LANES;
    kv::pdl_wait();
    kv::pdl_release();
    if (blockIdx.y == 0) check_lengths(a.bt, a.status);
    Unit x;
    if (!find_unit(a.bt, a.c, blockIdx.x, x)) return;
    if (!x.ok) {
        if (blockIdx.y == 0 && threadIdx.x == 0) kv::report(a.status);
        return;
    }
    for (int n = 0; n < kHeadsEach; n++) {
        const int head = (blockIdx.y * kHeadsEach + n) * kWarps + warp;
        if (head >= 2 * a.c.heads) return;
        const bool value = head >= a.c.heads;
        const int h = value ? head - a.c.heads : head;
        const uint8_t* codes = value ? a.vc : a.kc;
        uint4 w[ITER];
#pragma unroll
        for (int i = 0; i < ITER; i++) {
            const int slot = i * ROWS + row;
            if (slot >= x.s0 && slot < x.s1) w[i] = *reinterpret_cast<const uint4*>(codes + codes_at(a.c, x, slot, h) + 16 * j);
        }
        const float scale = pow2((int)*((value ? a.vs : a.ks) + scale_at(a.c, x, h)) - kBias);
#pragma unroll
        for (int i = 0; i < ITER; i++) {
            const int slot = i * ROWS + row;
            if (slot < x.s0 || slot >= x.s1) continue;
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            TO* to = static_cast<TO*>(value ? a.v : a.k) + (x.t0 + slot - x.s0) * (value ? a.ldv : a.ldk) + (long long)h * D + 16 * j;
            float f[2][8];
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const float2 lo = half2_floats(decode_lo(u[r])), hi = half2_floats(decode_hi(u[r]));
                float* g = &f[r / 2][4 * (r % 2)];
                g[0] = lo.x * scale; g[1] = lo.y * scale; g[2] = hi.x * scale; g[3] = hi.y * scale;
            }
            kv::store8(to, f[0]);
            kv::store8(to + 8, f[1]);
        }
    }
}

template <typename K, typename Args>
cudaError_t launch(K kernel, const Args& a, int64_t units, int heads, cudaStream_t s)
{
    const int64_t chunks = ceil_div(heads, kWarps * kHeadsEach);
    if (units > 0x7FFFFFFF || chunks > 65535) return cudaErrorInvalidConfiguration;
    return kv::launch_dependent(kernel, dim3((unsigned)units, (unsigned)chunks), kThreads, 0, s, a);
}

template <typename TI, int D>
cudaError_t append(const AppendArgs& a, int64_t units, cudaStream_t s)
{
    const int heads = a.heads_q + 2 * a.c.heads;
    if (a.bt.max_q == 1) return launch(k_kv8_append<TI, D, true>, a, units, (int)ceil_div(heads, 512 / D), s);
    return launch(k_kv8_append<TI, D, false>, a, units, heads, s);
}

template <int D>
cudaError_t append(const AppendArgs& a, int xt, int64_t units, cudaStream_t s)
{
    return xt == QG_T_F32 ? append<float, D>(a, units, s)
           : xt == QG_T_BF16 ? append<__nv_bfloat16, D>(a, units, s) : append<__half, D>(a, units, s);
}

template <int D>
cudaError_t read(const ReadArgs& a, int ot, int64_t units, cudaStream_t s)
{
    return ot == QG_T_F32    ? launch(k_kv8_read<float, D>, a, units, 2 * a.c.heads, s)
           : ot == QG_T_BF16 ? launch(k_kv8_read<__nv_bfloat16, D>, a, units, 2 * a.c.heads, s)
                             : launch(k_kv8_read<__half, D>, a, units, 2 * a.c.heads, s);
}

}  // namespace
}  // namespace kv8

qg_status launch_kv8_append(const qg_kv8_cache& cache, const qg_kv_batch& batch, const qg_head_norm* norm,
                            const qg_rope* rope, const void* q, int64_t ldq, int heads_q, const void* k, int64_t ldk,
                            const void* v, int64_t ldv, int xt, void* q_out, int64_t ldq_out, int qt, cudaStream_t s)
{
    kv8::AppendArgs a;
    a.bt = kv::make_batch(batch);
    a.c = kv8::make_cache(cache);
    a.kc = static_cast<uint8_t*>(cache.k); a.vc = static_cast<uint8_t*>(cache.v);
    a.ks = cache.k_scale; a.vs = cache.v_scale;
    a.q = q; a.k = k; a.v = v;
    a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldq_out = ldq_out;
    a.q_out = q_out;
    a.qt = qt;
    a.heads_q = heads_q;
    a.rope = rope ? rope->table : nullptr;
    a.at = rope ? rope->at : nullptr;
    a.positions = rope ? rope->positions : 0;
    a.rot = rope ? rope->dim : 0;
    a.interleaved = rope ? rope->interleaved != 0 : 0;
    a.norm = kv::make_norm(norm);
    a.status = device_status_ptr();
    const int64_t units = kv8::units_of(batch);
    const cudaError_t e = cache.head_dim == 128 ? kv8::append<128>(a, xt, units, s) : kv8::append<64>(a, xt, units, s);
    if (e != cudaSuccess) return cuda_fail(e, "qkv8_append launch");
    return QG_OK;
}

qg_status launch_kv8_read(const qg_kv8_cache& cache, const qg_kv_batch& batch, void* k, int64_t ldk, void* v, int64_t ldv,
                          int ot, cudaStream_t s)
{
    kv8::ReadArgs a;
    a.bt = kv::make_batch(batch);
    a.c = kv8::make_cache(cache);
    a.kc = static_cast<const uint8_t*>(cache.k); a.vc = static_cast<const uint8_t*>(cache.v);
    a.ks = cache.k_scale; a.vs = cache.v_scale;
    a.k = k; a.v = v;
    a.ldk = ldk; a.ldv = ldv;
    a.status = device_status_ptr();
    const int64_t units = kv8::units_of(batch);
    const cudaError_t e = cache.head_dim == 128 ? kv8::read<128>(a, ot, units, s) : kv8::read<64>(a, ot, units, s);
    if (e != cudaSuccess) return cuda_fail(e, "qkv8_read launch");
    return QG_OK;
}

}  // namespace qg
