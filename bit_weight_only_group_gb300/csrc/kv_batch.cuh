// What the paged-cache kernels share: the batch and cache as the kernels see
// them, the search for a token's sequence, and the bounds checks on lengths
// and page numbers (which set the status word instead of following them).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "qg_internal.h"

namespace qg {
namespace kv {

struct Batch {
    int B, T, max_q, max_kv, table_ld, prefix_len;
    const int* table;
    const int* kv_len;
    const int* cu_q;   // null: token b belongs to sequence b
    const int* prefix_table;
};

struct Cache {
    int num_pages, page_shift, heads, dim;
    long long page_stride, token_stride, head_stride;   // elements
};

inline Batch make_batch(const qg_kv_batch& b)
{
    return Batch{b.sequences, b.tokens, b.max_q, b.max_kv, b.table_ld, b.prefix_len,
                 b.table, b.kv_len, b.cu_q, b.prefix_table};
}

inline Cache make_cache(const qg_kv_cache& c)
{
    int sh = 0;
    while ((1 << sh) < c.page_size) sh++;
    return Cache{c.num_pages, sh, c.heads_kv, c.head_dim, c.page_stride, c.token_stride, c.head_stride};
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void report(int* status)
{
    if (status) atomicExch(status, (int)QG_ERR_DEVICE_STATUS);
}

// Token rows [t0, t1) of sequence b, cut to the array; false if they had to
// be, or if there are more than the bound.
__device__ __forceinline__ bool token_range(const Batch& bt, int b, int& t0, int& t1)
{
    if (!bt.cu_q) {
        t0 = b;
        t1 = min(b + 1, bt.T);
        return true;
    }
    const int from = __ldg(bt.cu_q + b), to = __ldg(bt.cu_q + b + 1);
    t0 = min(max(from, 0), bt.T);
    t1 = min(max(to, t0), bt.T);
    return t0 == from && t1 == to && t1 - t0 <= bt.max_q;
}

// Rows that belong to a sequence: [0, used_tokens).
__device__ __forceinline__ int used_tokens(const Batch& bt)
{
    return bt.cu_q ? min(max(__ldg(bt.cu_q + bt.B), 0), bt.T) : min(bt.B, bt.T);
}

// Own cached tokens of sequence b, cut to the bound; false if it had to be.
__device__ __forceinline__ bool own_length(const Batch& bt, int b, int& len)
{
    const int l = __ldg(bt.kv_len + b);
    len = min(max(l, 0), bt.max_kv);
    return l == len;
}

// Sequence of each lane's token (of a whole warp): the last b with cu_q[b] <= t.
// 32 bounds are loaded at once and searched by shuffles, so that up to 32
// sequences take one load and 256 four, one after another.
__device__ __forceinline__ int find_sequences(const Batch& bt, int t)
{
    if (!bt.cu_q) return min(t, bt.B - 1);
    const int lane = threadIdx.x & 31, step = (bt.B + 31) / 32;
    const int bound = lane * step < bt.B ? __ldg(bt.cu_q + lane * step) : 0x7FFFFFFF;
    int at = 0;
#pragma unroll
    for (int i = 16; i > 0; i /= 2)
        if (__shfl_sync(0xffffffffu, bound, at + i) <= t) at += i;
    int lo = at * step, hi = min(lo + step, bt.B);
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (__ldg(bt.cu_q + mid) <= t) lo = mid;
        else hi = mid;
    }
    return min(lo, bt.B - 1);
}

// fp32 pair -> two values of the cache's type in one word, rounded to nearest even.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Lets a kernel use `bytes` of dynamic shared memory, once per context.
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& done)
{
    const unsigned long long ctx = current_context_id();
    if (ctx && done.load(std::memory_order_acquire) == ctx) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.store(ctx, std::memory_order_release);
    return e;
}

// Launch that may start before the kernel ahead of it on the stream has
// finished (while dependent launch is on).  Every kernel launched this way
// waits for that kernel (pdl_wait) before it exits, so that completion stays
// transitive along the stream.
template <typename... KArgs, typename... Act>
inline cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                                    Act&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent_launch_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Act>(args)...);
}

}  // namespace kv
}  // namespace qg
