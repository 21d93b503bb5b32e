// ffn.cuh -- what the feed-forward block's tiled and few-token kernels share:
// the activations, packing to the 16-bit type, and the few-token entry point.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "host.h"

// A plan (the header's tgemm_ffn_t).
struct tgemm_ffn_s {
    int64_t width, hidden;
    int dtype, act;
    tg::Device dev;
    int pairs;  // CTA pairs resident at once
    int *d_status;
    unsigned long long watchdog_ns;
    int debug_stall;
};

namespace tg {

// The block's products: see ffn.cu.
enum Product : int { kUp = 0, kDown = 1, kDh = 2, kDx = 3, kDw = 4 };
enum Activation : int { kSilu = 0, kGelu = 1, kRelu = 2 };

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// act(g) and its derivative, of two values at once.  silu's 1 / (1 + exp(-g)) is
// formed with the hardware's approximate exp2 and reciprocal (about 2^-22
// relatively each, and |g| 2^-24 from the exponent's rounding): far below the
// 16-bit results' rounding.  Where exp(-g) overflows the reciprocal is 0, the
// limit.  gelu's normal distribution is exp(-g^2/2) R(|g|) below zero and 1 minus
// that above.  R(x) = exp(x^2/2) erfc(x / sqrt 2) / 2 is smooth, between 1/2 and
// 0.4 / x, and close to a polynomial in t = 1 / (1 + 0.265 x) without constant
// term; these seven coefficients are its best relative fit on 0 .. 14 (a linear
// program over 2000 points): 5.9e-7, and 1e-6 evaluated in fp32.  So the tail is
// right relatively, up to 1e-6 and the exponent's rounding of 1e-7 g^2, a hundredth
// of the 16-bit rounding down to g = -13, where the exponential (which the slope
// needs too) leaves fp32's range and the result becomes 0.
template <int ACT>
__device__ __forceinline__ void activate(F2 g, F2 &a, F2 &slope)
{
    const F2 one = f2(1.f);
    const float2 gs = split(g);
    if constexpr (ACT == kSilu) {
        const float2 t = split(g * f2(-1.44269504088896341f));
        const float2 q = split(f2(exp2_approx(t.x), exp2_approx(t.y)) + one);
        const F2 s = f2(rcp_approx(q.x), rcp_approx(q.y));
        a = g * s;
        slope = s * fma2(g, fma2(s, f2(-1.f), one), one);
    } else if constexpr (ACT == kGelu) {
        // R(|g|)
        const float2 d = split(fma2(f2(fabsf(gs.x), fabsf(gs.y)), f2(0.265f), one));
        const F2 t = f2(rcp_approx(d.x), rcp_approx(d.y));
        F2 q = fma2(t, f2(-0.0677719682f), f2(0.195213377f));
        q = fma2(q, t, f2(-0.0662704716f));
        q = fma2(q, t, f2(0.142422842f));
        q = fma2(q, t, f2(0.0829740727f));
        q = fma2(q, t, f2(0.107831668f));
        q = fma2(q, t, f2(0.105600187f));
        const float2 w = split(g * g * f2(-0.72134752044448170f));  // -g^2 / 2 in powers of 2
        const F2 e = f2(exp2_approx(w.x), exp2_approx(w.y));
        q = q * t * e;
        const float2 tail = split(q), rest = split(fma2(q, f2(-1.f), one));
        const F2 cdf = f2(gs.x < 0.f ? tail.x : rest.x, gs.y < 0.f ? tail.y : rest.y);
        a = g * cdf;
        slope = fma2(g * f2(0.39894228040143268f), e, cdf);
    } else {
        a = f2(gs.x <= 0.f ? 0.f : gs.x, gs.y <= 0.f ? 0.f : gs.y);  // a NaN comes through
        slope = f2(gs.x <= 0.f ? 0.f : 1.f, gs.y <= 0.f ? 0.f : 1.f);
    }
}

// For one value.
template <int ACT>
__device__ __forceinline__ void activate(float g, float &a, float &slope)
{
    F2 a2, s2;
    activate<ACT>(f2(g), a2, s2);
    a = split(a2).x;
    slope = split(s2).x;
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

__device__ __forceinline__ uint32_t pack2(F2 v, int bf16)
{
    const float2 s = split(v);
    return pack2(s.x, s.y, bf16);
}

__device__ __forceinline__ float2 unpack2(uint32_t w, int bf16)
{
    if (bf16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// One matrix: `rows` x `cols` elements, `ld` from row to row.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
};

// A product: A (m x k), B (n x k) and output matrices by problem (or segment,
// or projection), as FfnParams lists them.
struct Job {
    int prod, problems;
    int64_t k;          // reduction length (of one segment)
    int na, nb, nc;     // matrices given
    Mat A[3], B[3], C[3];
    const void *g, *u;  // Dh: the projections, as C's matrices
    // Dw launched right after Dx: it reads nothing that Dx writes, and Dx lets it
    // start only once Dh has finished (each of Dx's CTAs waits for Dh before it
    // releases its dependents), so it runs beside Dx's last tiles and waits for Dx
    // at its own end, so that what follows finds both finished.
    bool beside;
    // Dx and Dw of one call: their cuts weigh the share of the SMs that they leave
    // to each other (kShare).
    bool shared;
};

// How much a shared product's share of all SMs' time counts beside its own time.
constexpr double kShare = 1.33;

constexpr int kBlockK = 64;                    // reduction elements per slot: one 128-byte swizzle row
constexpr uint32_t kSlot = 128 * kBlockK * 2;  // bytes of one operand's slot in one CTA: 128 rows
constexpr uint32_t kPanel = 64 * kBlockK * 2;  // an MN-major box: 64 columns x 64 reduction rows
// Shared-memory matrix descriptor (layout as in tgemm.cu), 128-byte swizzle,
// groups of 8 swizzle rows 1024 bytes apart.  A K-major tile's swizzle row is
// one operand row's 64 reduction elements; an MN-major tile's is one reduction
// index's 64 columns, and the next 64 columns follow one panel further on (the
// leading byte offset).
__device__ __forceinline__ uint64_t ffn_desc(uint32_t addr, bool mn)
{
    const uint32_t lead = mn ? kPanel >> 4 : 1u;
    const uint32_t lo = ((addr >> 4) & 0x3FFFu) | (lead << 16);
    const uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    return (uint64_t(hi) << 32) | lo;
}

// A product cut up for few tokens or few tiles (ffn_few.cu): the best cut with
// its estimated SM cycles, and the launch.
struct FewShape {
    int64_t tiles;  // of all problems
    int ranks, n, kb_each;
};
FewShape ffn_few_shape(const tgemm_ffn_s *f, const Job &j, double *cycles);
int ffn_few_product(tgemm_ffn_s *f, const Job &j, const FewShape &c, cudaStream_t s);

// Most tokens that ffn_rows_forward takes.
constexpr int kRowsTokens = 8;

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
