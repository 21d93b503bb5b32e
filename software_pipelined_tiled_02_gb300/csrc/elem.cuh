// elem.cuh -- element types of the row-wise operators: 16-byte vectors of
// fp32, fp16 or bf16 values, read to and rounded from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

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

// ---------------------------------------------------------------- pairs of fp32 values

// Two fp32 values in one 64-bit register pair: one instruction adds, multiplies
// or multiply-adds both, each rounded as by itself.
struct F2 {
    uint64_t v;
};

__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
__device__ __forceinline__ float2 split(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum2(F2 a)
{
    const float2 r = split(a);
    return r.x + r.y;
}

// The values of a 16-byte vector as pairs, and back (rounded to nearest even).
template <class T>
__device__ __forceinline__ void unpack16(const uint4 &q, F2 (&f)[8 / sizeof(T)])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
        f[0] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        f[1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            } else {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                f[i] = f2(v.x, v.y);
            }
        }
    }
}

template <class T>
__device__ __forceinline__ uint4 pack16(const F2 (&f)[8 / sizeof(T)])
{
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
        const float2 a = split(f[0]), b = split(f[1]);
        w[0] = __float_as_uint(a.x);
        w[1] = __float_as_uint(a.y);
        w[2] = __float_as_uint(b.x);
        w[3] = __float_as_uint(b.y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = split(f[i]);
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(v.x, v.y);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace tg
