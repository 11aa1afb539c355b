// Appending keys and values to the paged cache, the position rotation applied
// on the way; the queries are turned in the same pass.
//
// For a rotated pair (a, c) with the position's cosine and sine:
//     a' = a cos - c sin,  c' = c cos + a sin,
// in fp32, rounded once to the cache's type.
//
// Bound by HBM: every value is read and written once and the arithmetic is a
// few operations a value.  One CTA takes one token, so that the search for
// its sequence and its page, a chain of dependent loads, is made once per 160
// to 1280 16-value tasks and runs under the loads of the token's values,
// which are issued first.  A thread's task is 16 values of one head: the two
// 8-value runs (16 bytes each) that hold 8 pairs, so that each run is one
// vector load and one vector store.
#include "kv_batch.cuh"

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
    int* status;
};

constexpr int kPerThread = 2;   // tasks of a thread whose loads are in flight together

template <typename T> struct Run8 { uint4 w; };                 // 8 values of 16 bits
template <> struct Run8<float> { float4 w[2]; };

template <typename T> __device__ __forceinline__ Run8<T> load8(const T* p)
{
    Run8<T> r;
    if constexpr (sizeof(T) == 4) {
        r.w[0] = __ldg(reinterpret_cast<const float4*>(p));
        r.w[1] = __ldg(reinterpret_cast<const float4*>(p) + 1);
    } else {
        r.w = __ldg(reinterpret_cast<const uint4*>(p));
    }
    return r;
}

template <typename T> __device__ __forceinline__ void to_float(const Run8<T>& r, float (&f)[8])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            f[4 * i] = r.w[i].x; f[4 * i + 1] = r.w[i].y; f[4 * i + 2] = r.w[i].z; f[4 * i + 3] = r.w[i].w;
        }
    } else {
        const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 v;
            if constexpr (std::is_same<T, __half>::value) v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            else v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

template <typename T> __device__ __forceinline__ void store8(T* p, const float (&f)[8])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                                              pack2<T>(f[6], f[7]));
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(512) k_kv_append(const __grid_constant__ AppendArgs a)
{
    pdl_wait();      // the values, lengths and tables may come from the kernel just before
    pdl_release();
    const int t = blockIdx.x;
    const int per_head = a.c.dim / 16, hq = a.heads_q, hk = a.c.heads;
    const int tasks = (hq + 2 * hk) * per_head, turned = a.rope ? a.rot / 16 : 0;
    const int used = used_tokens(a.bt);   // waited for only after the values' loads are under way

    // of a task: its head's values, and where in the head its two runs are
    auto place = [&](int task, int& head, int& i0, int& i1, bool& turn) {
        head = task / per_head;
        const int j = task - head * per_head;
        turn = head < hq + hk && j < turned;
        i0 = turn && !a.interleaved ? 8 * j : 16 * j;
        i1 = turn && !a.interleaved ? a.rot / 2 + 8 * j : 16 * j + 8;
    };
    int b = -1, page = -1, in_page = 0;
    long long at = -1;
    for (int base = 0; base < tasks; base += kPerThread * (int)blockDim.x) {
        Run8<TI> x0[kPerThread], x1[kPerThread];
#pragma unroll
        for (int u = 0; u < kPerThread; u++) {
            const int task = base + u * (int)blockDim.x + (int)threadIdx.x;
            if (task < tasks) {
                int head, i0, i1;
                bool turn;
                place(task, head, i0, i1, turn);
                const TI* src = head < hq ? static_cast<const TI*>(a.q) + t * a.ldq + (long long)head * a.c.dim
                                : head < hq + hk
                                    ? static_cast<const TI*>(a.k) + t * a.ldk + (long long)(head - hq) * a.c.dim
                                    : static_cast<const TI*>(a.v) + t * a.ldv + (long long)(head - hq - hk) * a.c.dim;
                x0[u] = load8(src + i0);
                x1[u] = load8(src + i1);
            }
        }
        if (base == 0) {   // the token's sequence, page and position
            if (t >= used) return;
            b = find_sequence(a.bt, t);
            int t0, t1, len;
            token_range(a.bt, b, t0, t1);
            bool ok = own_length(a.bt, b, len) && t1 - t0 <= a.bt.max_q;
            const int own = len - (t1 - t) ;   // len - n + i
            if (own >= 0 && own < len) {
                const int e = own >> a.c.page_shift;
                const int p = e < a.bt.table_ld ? __ldg(a.bt.table + (long long)b * a.bt.table_ld + e) : -1;
                if (p >= 0 && p < a.c.num_pages) page = p;
                in_page = own & ((1 << a.c.page_shift) - 1);
            }
            ok = ok && page >= 0;
            if (a.rope) {
                at = a.at ? (long long)__ldg(a.at + t) : (long long)a.bt.prefix_len + own;
                if (at < 0 || at >= a.positions) {
                    at = -1;
                    ok = false;
                }
            } else {
                at = 0;
            }
            if (!ok && threadIdx.x == 0) report(a.status);
        }
        if (at < 0) return;
#pragma unroll
        for (int u = 0; u < kPerThread; u++) {
            const int task = base + u * (int)blockDim.x + (int)threadIdx.x;
            if (task >= tasks) continue;
            int head, i0, i1;
            bool turn;
            place(task, head, i0, i1, turn);
            if (head >= hq && page < 0) continue;
            float f0[8], f1[8];
            to_float(x0[u], f0);
            to_float(x1[u], f1);
            if (turn) {
                // pairs 8j .. 8j + 7 of the head, in f0 and f1, or adjacent
                const int j = task - head * per_head;
                const float* row = a.rope + at * a.rot + 8 * j;
                float cs[8], sn[8];
                to_float(load8(row), cs);
                to_float(load8(row + a.rot / 2), sn);
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float p = f0[2 * i], r = f0[2 * i + 1], p1 = f1[2 * i], r1 = f1[2 * i + 1];
                        f0[2 * i] = p * cs[i] - r * sn[i];
                        f0[2 * i + 1] = r * cs[i] + p * sn[i];
                        f1[2 * i] = p1 * cs[4 + i] - r1 * sn[4 + i];
                        f1[2 * i + 1] = r1 * cs[4 + i] + p1 * sn[4 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float p = f0[i], r = f1[i];
                        f0[i] = p * cs[i] - r * sn[i];
                        f1[i] = r * cs[i] + p * sn[i];
                    }
                }
            }
            TO* dst;
            if (head < hq) {
                dst = static_cast<TO*>(a.q_out) + t * a.ldq_out + (long long)head * a.c.dim;
            } else {
                const bool key = head < hq + hk;
                dst = static_cast<TO*>(key ? a.kc : a.vc) + (long long)page * a.c.page_stride +
                      (long long)in_page * a.c.token_stride + (long long)(head - hq - (key ? 0 : hk)) * a.c.head_stride;
            }
            store8(dst + i0, f0);
            store8(dst + i1, f1);
        }
    }
}

template <typename TI, typename TO>
cudaError_t launch(const AppendArgs& a, cudaStream_t s)
{
    const int tasks = (a.heads_q + 2 * a.c.heads) * (a.c.dim / 16);
    const int threads = (int)std::min<int64_t>(512, ceil_div(ceil_div(tasks, kPerThread), 32) * 32);
    return launch_dependent(k_kv_append<TI, TO>, dim3((unsigned)a.bt.T), threads, 0, s, a);
}

template <typename TO>
cudaError_t by_input(const AppendArgs& a, int xt, cudaStream_t s)
{
    switch (xt) {
        case QG_T_F32: return launch<float, TO>(a, s);
        case QG_T_BF16: return launch<__nv_bfloat16, TO>(a, s);
        default: return launch<__half, TO>(a, s);
    }
}

}  // namespace
}  // namespace kv

qg_status launch_kv_append(const qg_kv_cache& cache, const qg_kv_batch& batch, const qg_rope* rope, const void* q,
                           int64_t ldq, int heads_q, const void* k, int64_t ldk, const void* v, int64_t ldv, int xt,
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
    a.status = device_status_ptr();
    const cudaError_t e = cache.dtype == QG_T_BF16 ? kv::by_input<__nv_bfloat16>(a, xt, s)
                                                   : kv::by_input<__half>(a, xt, s);
    if (e != cudaSuccess) return cuda_fail(e, "qkv_append launch");
    return QG_OK;
}

}  // namespace qg
