// ffn.cuh -- what the feed-forward block's tiled and few-token kernels share:
// the activations, packing to the 16-bit type, and the few-token entry point.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

enum Activation : int { kSilu = 0, kGelu = 1, kRelu = 2 };

// act(g) and its derivative.
template <int ACT>
__device__ __forceinline__ void activate(float g, float &a, float &slope)
{
    if constexpr (ACT == kSilu) {
        const float s = __fdividef(1.f, 1.f + __expf(-g));
        a = g * s;
        slope = s * (1.f + g * (1.f - s));
    } else if constexpr (ACT == kGelu) {
        const float cdf = 0.5f * (1.f + erff(g * 0.70710678118654752f));
        a = g * cdf;
        slope = cdf + g * 0.39894228040143268f * __expf(-0.5f * g * g);
    } else {
        a = g <= 0.f ? 0.f : g;  // a NaN comes through
        slope = g <= 0.f ? 0.f : 1.f;
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int bf16)
{
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float2 unpack2(uint32_t w, int bf16)
{
    if (bf16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Most tokens that ffn_rows_forward takes.
constexpr int kRowsTokens = 32;

// The forward pass for 1 .. kRowsTokens tokens (ffn_rows.cu).  Pointers and
// leading dimensions have been checked by the caller.
struct FfnRows {
    int tokens;
    int64_t width, hidden, ldx, ld_gate, ld_up, ld_down, ldy;
    const void *x, *w_gate, *w_up, *w_down;
    void *y, *g, *u, *h;  // g and u may be NULL
    int bf16, act;
};
int ffn_rows_forward(const FfnRows &a, cudaStream_t s);

}  // namespace tg
