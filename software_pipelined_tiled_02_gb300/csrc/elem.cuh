// elem.cuh -- element types of the row-wise operators: 16-byte vectors of
// fp32, fp16 or bf16 values, read to and rounded from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace tg {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements as they lie in memory: one element, or 16 bytes.
template <class T, int V>
struct Pack {
    static_assert(V == 1 || V * sizeof(T) == 16, "one element or 16 bytes");
    union {
        T v[V];
        uint4 q;
    };
    __device__ Pack() {}
};
template <class T>
struct Pack<T, 1> {
    T v[1];
};

template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p)
{
    Pack<T, V> r;
    if constexpr (V == 1)
        r.v[0] = *p;
    else
        r.q = *reinterpret_cast<const uint4 *>(p);
    return r;
}

template <class T, int V>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &r)
{
    if constexpr (V == 1)
        *p = r.v[0];
    else
        *reinterpret_cast<uint4 *>(p) = r.q;
}

// V weights at index i of an array of type T or (f32) of fp32, to fp32.
template <class T, int V>
__device__ __forceinline__ void load_weights(const void *w, int64_t i, bool f32, float (&out)[V])
{
    if (f32) {
        const float *p = static_cast<const float *>(w) + i;
        if constexpr (V == 1) {
            out[0] = *p;
        } else {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                const float4 q = *reinterpret_cast<const float4 *>(p + e);
                out[e] = q.x;
                out[e + 1] = q.y;
                out[e + 2] = q.z;
                out[e + 3] = q.w;
            }
        }
    } else {
        const Pack<T, V> q = load_pack<T, V>(static_cast<const T *>(w) + i);
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = to_f32(q.v[e]);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace tg
