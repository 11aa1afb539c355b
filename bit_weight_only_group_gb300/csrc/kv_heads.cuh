// Runs of a head's values in fp32 as the appending kernels hold them, and the
// norm of a head.
#pragma once

#include <type_traits>

#include "kv_batch.cuh"

namespace qg {
namespace kv {

template <typename T> struct Run8 { uint4 w; };                 // 8 values of 16 bits
template <> struct Run8<float> { float4 w[2]; };

template <typename T> __device__ __forceinline__ Run8<T> load8(const T* p)
{
    return *reinterpret_cast<const Run8<T>*>(p);
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

template <> __device__ __forceinline__ void store8<float>(float* p, const float (&f)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Eight pairs of a head turned: (f0[i], f1[i]), or, interleaved, neighbours in f0 and then in f1.
__device__ __forceinline__ void turn16(float (&f0)[8], float (&f1)[8], const float (&cs)[8], const float (&sn)[8],
                                       bool interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float c = f0[2 * i], d = f0[2 * i + 1], e = f1[2 * i], f = f1[2 * i + 1];
            f0[2 * i] = c * cs[i] - d * sn[i];
            f0[2 * i + 1] = d * cs[i] + c * sn[i];
            f1[2 * i] = e * cs[4 + i] - f * sn[4 + i];
            f1[2 * i + 1] = f * cs[4 + i] + e * sn[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float c = f0[i], d = f1[i];
            f0[i] = c * cs[i] - d * sn[i];
            f1[i] = d * cs[i] + c * sn[i];
        }
    }
}

// Weights of the norms of queries and keys (qg_head_norm; null: not normed).
struct Norm {
    const void *q, *k;
    int type;
    float eps;
};

inline Norm make_norm(const qg_head_norm* n) { return n ? Norm{n->q, n->k, n->dtype, n->eps} : Norm{nullptr, nullptr, 0, 0.0f}; }

// Weight i of the keys' or the queries' norm in fp32 (0 where there is none).
__device__ __forceinline__ float norm_weight(const Norm& n, bool key, int i)
{
    const void* p = key ? n.k : n.q;
    if (!p) return 0.0f;
    if (n.type == QG_T_F32) return static_cast<const float*>(p)[i];
    if (n.type == QG_T_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

// The weights of both norms in shared memory as the lanes of a head read them, 16 bytes at a time without a conflict:
// [queries, keys][quarter of a lane's 16 weights][lane][4], the lane's two runs of 8 where the rotation wants them (rot 0:
// there is none).  (In the order of the head eight lanes met four banks: 8192 tokens 73.4 us, 69 to 71 so.)  By at least 32 LANES
// threads.
template <int LANES>
__device__ __forceinline__ void stage_weights(float4* w, const Norm& n, int rot, bool interleaved)
{
    const int t = threadIdx.x;
    if (t >= 32 * LANES) return;
    const int j = t / 4 % LANES, c = t / (4 * LANES) % 4;
    const bool apart = j < rot / 16 && !interleaved;
    const int run = c < 2 ? (apart ? 8 * j : 16 * j) : (apart ? rot / 2 + 8 * j : 16 * j + 8);
    reinterpret_cast<float*>(w)[t] = norm_weight(n, t >= 16 * LANES, run + 4 * (c & 1) + t % 4);
}

// x w / sqrt(mean x^2 + eps) over a head of D values, 16 a lane over LANES neighbouring lanes; lanes of other heads need
// not take part.  w: the lane's staged weights, LANES apart.
template <int LANES, int D>
__device__ __forceinline__ void norm_head(float (&f0)[8], float (&f1)[8], const float4* w, float eps)
{
    const uint32_t mask = ((1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        s0 = fmaf(f0[i], f0[i], s0);
        s1 = fmaf(f1[i], f1[i], s1);
    }
    s0 += s1;
#pragma unroll
    for (int i = LANES / 2; i > 0; i /= 2) s0 += __shfl_xor_sync(mask, s0, i);
    const float r = rsqrtf(fmaf(s0, 1.0f / D, eps));
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 a = w[i / 4 * LANES], b = w[(2 + i / 4) * LANES];
        f0[i] *= r * a.x; f0[i + 1] *= r * a.y; f0[i + 2] *= r * a.z; f0[i + 3] *= r * a.w;
        f1[i] *= r * b.x; f1[i + 1] *= r * b.y; f1[i + 2] *= r * b.z; f1[i + 3] *= r * b.w;
    }
}

}  // namespace kv
}  // namespace qg
