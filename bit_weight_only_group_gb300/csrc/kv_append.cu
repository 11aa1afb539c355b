// Appending keys and values to the paged cache, the position rotation applied
// on the way; the queries are turned in the same pass.
//
// For a rotated pair (a, c) with the position's cosine and sine:
//     a' = a cos - c sin,  c' = c cos + a sin,
// in fp32, rounded once to the cache's type.  Where queries and keys are normed
// (a form of the kernel of its own) x becomes x w / sqrt(mean x^2 + eps) first:
// the threads of a head sum their squares by shuffles, and the weights lie in
// shared memory in fp32 (8192 tokens of 64 + 2 x 8 heads 69 to 71 us, 58.3 without
// norms).
//
// Bound by HBM: every value is read and written once and the arithmetic is a
// few operations a value.  A CTA works through units (a token, or some heads of
// one where it has many).  The values of its next units come by bulk copies
// into a ring in shared memory while one is worked on; a warp of its own finds
// the places of the next 32 units, a chain of dependent loads; and the next
// token's cosines and sines are loaded with the place found before.  A thread
// takes 16 values of a head: the two 8-value runs (16 bytes each) that hold 8
// pairs.  8192 tokens of 64 + 2 x 8 heads of 128 (bf16, 340 MB): 58.7 us, 5.8 TB/s;
// a plain copy of as much takes 55.5.  With a CTA a token and its place found
// by itself 66 us (1.5 us of dependent loads a token, whatever was in flight).
// One token 4.0 us, 256 tokens 4.8 us, one launch after another in a graph.
// fp32 values into an fp16 cache are further from the bytes' time: 778 tokens of
// 32 + 2 x 32 heads (58 MB) 17.9 us, 3.2 TB/s.  A CTA has about five units there
// (two a token), too few to hide the launch's start and end (the 4.0 us of one
// token) and the first places; what the rest waits for has not been measured.
#include "kv_heads.cuh"
#include "ptx.cuh"

#include <algorithm>
#include <utility>

namespace qg {
namespace kv {
namespace {

struct AppendArgs {
    Batch bt;
    Cache c;
    void *kc, *vc;
    const void *q, *k, *v;
    long long ldq, ldk, ldv, ldq_out;
    void* q_out;
    int heads_q;
    const float* rope;   // null: no rotation
    const int* at;
    int positions, rot, interleaved;
    Norm norm;
    int* status;
};

constexpr int kWorkers = 256, kThreads = kWorkers + 32;   // the last warp finds places; two CTAs an SM
constexpr int kPlaces = 64;                   // two rounds of a warp's
constexpr int kStages = 4, kStageBytes = 24 * 1024;   // at most

// Where a token goes.
struct Place {
    int page, in_page;   // page -1: not cached
    long long at;        // its row of the rotation table; -1: not written at all
};

// The places of each lane's token, of a whole warp; there: the lane has one.
__device__ __forceinline__ Place find_place(const AppendArgs& a, int t, bool there)
{
    Place p{-1, 0, 0};
    const int b = find_sequences(a.bt, t);
    if (!there) return p;
    int t0, t1, len;
    // a length or an offset outside its bound says nothing of where the token belongs: it is not cached, so that what is
    // stays
    bool ok = token_range(a.bt, b, t0, t1) && t >= t0 && t < t1;
    ok = own_length(a.bt, b, len) && ok;
    const int own = len - (t1 - t);   // len - n + i
    if (ok && own >= 0 && own < len) {
        const int e = own >> a.c.page_shift;
        const int page = e < a.bt.table_ld ? __ldg(a.bt.table + (long long)b * a.bt.table_ld + e) : -1;
        if (page >= 0 && page < a.c.num_pages) p.page = page;
        p.in_page = own & ((1 << a.c.page_shift) - 1);
    }
    ok = ok && p.page >= 0;
    if (a.rope) {
        p.at = a.at ? (long long)__ldg(a.at + t) : (long long)a.bt.prefix_len + own;
        if (p.at < 0 || p.at >= a.positions) {
            p.at = -1;
            ok = false;
        }
    }
    if (!ok) report(a.status);
    return p;
}

template <typename TI, typename TO, int D, bool NORM>
__global__ void __launch_bounds__(kThreads, 2) k_kv_append(const __grid_constant__ AppendArgs a, int chunks, int stages)
{
    constexpr int per_head = D / 16, chunk_heads = kStageBytes / (D * (int)sizeof(TI));
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ Place places[kPlaces];
    __shared__ float4 weights[NORM ? 8 * per_head : 1];   // of queries and keys (stage_weights)
    __shared__ __align__(8) uint64_t arrived[kStages];
    const uint32_t bars = ptx::smem_u32(arrived);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; i++) ptx::mbar_init(bars + 8 * i, 1);
        ptx::fence_mbar_init();
    }
    pdl_wait();      // the values, lengths and tables may come from the kernel just before
    pdl_release();
    __syncthreads();
    // units: tokens times chunks of the heads (query heads, then key heads, then value heads)
    const int hq = a.heads_q, hk = a.c.heads, heads = hq + 2 * hk;
    const long long units = (long long)used_tokens(a.bt) * chunks;
    const long long stride = gridDim.x;
    auto load = [&](long long unit, int stage) {
        if (unit >= units || threadIdx.x != kWorkers) return;
        const int t = (int)(unit / chunks), lo = (int)(unit % chunks) * chunk_heads, hi = min(lo + chunk_heads, heads);
        ptx::mbar_expect_tx(bars + 8 * stage, (uint32_t)((hi - lo) * D * (int)sizeof(TI)));
        auto part = [&](const void* base, long long ld, int from, int to) {   // heads [from, to) of one array
            const int x = max(lo, from), y = min(hi, to);
            if (x < y)
                ptx::bulk_load(ptx::smem_u32(ring + stage * kStageBytes + (x - lo) * D * (int)sizeof(TI)),
                               static_cast<const TI*>(base) + t * ld + (x - from) * D, (uint32_t)((y - x) * D * (int)sizeof(TI)),
                               bars + 8 * stage);
        };
        part(a.q, a.ldq, 0, hq);
        part(a.k, a.ldk, hq, hq + hk);
        part(a.v, a.ldv, hq + hk, heads);
    };
    // the places of the CTA's units number `from` to `from` + 31
    auto find = [&](int from) {
        if (threadIdx.x < kWorkers) return;
        const int n = from + (int)threadIdx.x - kWorkers;
        const long long unit = blockIdx.x + n * stride;
        const Place p = find_place(a, (int)(min(unit, units - 1) / chunks), unit < units);
        places[n % kPlaces] = p;
    };
    for (int i = 0; i < stages; i++) load(blockIdx.x + i * stride, i);
    if (blockIdx.x >= units) return;   // fewer tokens in use than rows
    // a thread keeps its 16 values' place in the head, and with it its cosines and sines, for all its heads
    const int j = threadIdx.x % per_head, first = threadIdx.x / per_head;
    constexpr int step = kWorkers / per_head;
    const bool turn = a.rope && j < a.rot / 16;
    // where in a turned head the two runs are, and in a value head
    const int t0 = turn && !a.interleaved ? 8 * j : 16 * j, t1 = turn && !a.interleaved ? a.rot / 2 + 8 * j : 16 * j + 8;
    if constexpr (NORM) stage_weights<per_head>(weights, a.norm, a.rot, a.interleaved);
    find(0);
    __syncthreads();

    const int v0 = 16 * j, v1 = 16 * j + 8;
    auto angles = [&](const Place& p, float (&cs)[8], float (&sn)[8]) {   // pairs 8j .. 8j + 7 of the head
        if (!turn || p.at < 0) return;
        const float* row = a.rope + p.at * a.rot + 8 * j;
        to_float(load8(row), cs);
        to_float(load8(row + a.rot / 2), sn);
    };
    int stage = 0, n = 0;   // n: units done
    uint32_t phase = 0;
    float cs[8], sn[8], next_cs[8], next_sn[8];
    Place p = places[0];
    angles(p, next_cs, next_sn);
    for (long long unit = blockIdx.x; unit < units; unit += stride) {
        const int t = (int)(unit / chunks), lo = (int)(unit % chunks) * chunk_heads, hi = min(lo + chunk_heads, heads);
        p = places[n % kPlaces];
#pragma unroll
        for (int i = 0; i < 8; i++) { cs[i] = next_cs[i]; sn[i] = next_sn[i]; }
        // places are found 32 at a time, while the first of the 32 before them is worked on
        if (n % 32 == 0 && unit + 32 * stride < units) find(n + 32);
        n++;
        if (unit + stride < units) angles(places[n % kPlaces], next_cs, next_sn);
        bool ok = ptx::mbar_wait(bars + 8 * stage, phase);
        if constexpr (NORM) ok = __all_sync(0xffffffffu, ok);   // a head's threads shuffle together or not at all
        const TI* x = reinterpret_cast<const TI*>(ring + stage * kStageBytes);
        const long long cached = (long long)p.page * a.c.page_stride + (long long)p.in_page * a.c.token_stride;
        for (int head = lo + first; threadIdx.x < kWorkers && ok && p.at >= 0 && head < hi; head += step) {
            if (head >= hq && p.page < 0) continue;
            const bool value = head >= hq + hk;
            const int i0 = value ? v0 : t0, i1 = value ? v1 : t1;
            float f0[8], f1[8];
            to_float(load8(x + (head - lo) * D + i0), f0);
            to_float(load8(x + (head - lo) * D + i1), f1);
            if constexpr (NORM) {
                const bool key = head >= hq;
                if (!value && (key ? a.norm.k : a.norm.q)) norm_head<per_head, D>(f0, f1, weights + key * 4 * per_head + j, a.norm.eps);
            }
            if (turn && !value) turn16(f0, f1, cs, sn, a.interleaved);
            TO* dst = head < hq ? static_cast<TO*>(a.q_out) + t * a.ldq_out + head * D
                                : static_cast<TO*>(value ? a.vc : a.kc) + cached +
                                      (long long)(head - hq - (value ? hk : 0)) * a.c.head_stride;
            store8(dst + i0, f0);
            store8(dst + i1, f1);
        }
        // the stage has been read, and the next place is there
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0 && a.status) atomicExch(a.status, (int)QG_ERR_TIMEOUT);
            // no copy is in flight when the CTA leaves
            for (int i = 0; i < stages && unit + i * stride < units; i++) {
                ptx::mbar_wait(bars + 8 * stage, phase);
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            return;
        }
        load(unit + stages * stride, stage);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
}

template <typename TI, typename TO, int D, bool NORM>
cudaError_t launch(const AppendArgs& a, cudaStream_t s)
{
    auto kernel = k_kv_append<TI, TO, D, NORM>;
    const int heads = a.heads_q + 2 * a.c.heads, chunks = (int)ceil_div(heads, kStageBytes / (D * (int)sizeof(TI)));
    const int64_t units = (int64_t)a.bt.T * chunks, grid = std::min<int64_t>(units, 2 * num_sms());
    const int stages = (int)std::min<int64_t>(kStages, ceil_div(units, grid)), smem = stages * kStageBytes;
    if (stages > 1) {   // with the places, above the 48 KB that need no attribute
        static std::atomic<unsigned long long> done{0};
        const cudaError_t e = allow_smem(kernel, kStages * kStageBytes, done);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kernel, dim3((unsigned)grid), kThreads, smem, s, a, chunks, stages);
}

template <typename TO, int D, bool NORM>
cudaError_t by_input(const AppendArgs& a, int xt, cudaStream_t s)
{
    switch (xt) {
        case QG_T_F32: return launch<float, TO, D, NORM>(a, s);
        case QG_T_BF16: return launch<__nv_bfloat16, TO, D, NORM>(a, s);
        default: return launch<__half, TO, D, NORM>(a, s);
    }
}

template <typename TO>
cudaError_t by_dim(const AppendArgs& a, int xt, cudaStream_t s)
{
    if (a.norm.q || a.norm.k)
        return a.c.dim == 128 ? by_input<TO, 128, true>(a, xt, s) : by_input<TO, 64, true>(a, xt, s);
    return a.c.dim == 128 ? by_input<TO, 128, false>(a, xt, s) : by_input<TO, 64, false>(a, xt, s);
}

}  // namespace
}  // namespace kv

qg_status launch_kv_append(const qg_kv_cache& cache, const qg_kv_batch& batch, const qg_head_norm* norm,
                           const qg_rope* rope, const void* q, int64_t ldq, int heads_q, const void* k, int64_t ldk, const void* v, int64_t ldv, int xt,
                           void* q_out, int64_t ldq_out, cudaStream_t s)
{
    kv::AppendArgs a;
    a.bt = kv::make_batch(batch);
    a.c = kv::make_cache(cache);
    a.kc = cache.k; a.vc = cache.v;
    a.q = q; a.k = k; a.v = v;
    a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldq_out = ldq_out;
    a.q_out = q_out;
    a.heads_q = heads_q;
    a.rope = rope ? rope->table : nullptr;
    a.at = rope ? rope->at : nullptr;
    a.positions = rope ? rope->positions : 0;
    a.rot = rope ? rope->dim : 0;
    a.interleaved = rope ? rope->interleaved != 0 : 0;
    a.norm = kv::make_norm(norm);
    a.status = device_status_ptr();
    const cudaError_t e = cache.dtype == QG_T_BF16 ? kv::by_dim<__nv_bfloat16>(a, xt, s)
                                                   : kv::by_dim<__half>(a, xt, s);
    if (e != cudaSuccess) return cuda_fail(e, "qkv_append launch");
    return QG_OK;
}

}  // namespace qg
