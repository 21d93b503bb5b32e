// ffn_rows.cu -- the gated feed-forward block's forward pass for one to eight
// tokens and few weights, for GB300 (sm_103a).
//
// Such a pass is short: what counts is how soon the weights start to move and
// how many requests are on their way.  The weights go from memory straight into
// the registers of tensor-core fragments, without tensor maps, barriers or
// tensor memory to set up.  The sum over k is the same in any order, so a
// lane's 16-byte load of 8 consecutive k of one weight row serves as two steps'
// fragments, as long as the tokens' values are taken at the same k.
//
// One m16n8k16 step takes 16 weight rows and 8 tokens.  In the first kernel
// rows 0-7 are gate rows and rows 8-15 the same hidden units' up rows, so a
// lane ends up with g and u of the same unit and token.  The warps of a CTA
// share out k and add their sums in warp order.

#include "elem.cuh"
#include "ffn.cuh"
#include "host.h"
#include "ptx.cuh"

namespace tg {

constexpr int kRowWarps = 8;
constexpr int kChunk = 128;  // k per warp and step: four 16-byte loads a lane and weight row

// 16 bytes of a weight, which is not read again: kept out of L1.
__device__ __forceinline__ uint4 load_stream(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 16 bytes of the tokens' values, read once by each warp: from L2.
__device__ __forceinline__ uint4 load_tokens(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// C += A . B^T for 16 rows, 8 tokens and 16 k: a0, a2 of row g, a1, a3 of row
// g + 8, b0, b1 of token g (g = lane / 4).
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, int bf16)
{
    if (bf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sums over this warp's share of k (chunks warp, warp + 8, ...) for 16 weight
// rows and 8 tokens.  `lo`, `hi` and `x` point at this lane's weight rows g and
// g + 8 and its token g (NULL: past the matrix, zeros).
__device__ __forceinline__ void stream_k(const uint16_t *lo, const uint16_t *hi, const uint16_t *x, int64_t k_len,
                                         int bf16, float (&c)[4])
{
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t k0 = int64_t(warp) * kChunk; k0 < k_len; k0 += kRowWarps * kChunk) {
        uint4 a[4], b[4], t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = k0 + i * 32 + (lane % 4) * 8;
            const bool in = k < k_len;
            a[i] = in && lo ? load_stream(lo + k) : zero;
            b[i] = in && hi ? load_stream(hi + k) : zero;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = k0 + i * 32 + (lane % 4) * 8;
            t[i] = k < k_len && x ? load_tokens(x + k) : zero;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mma_16816(c, a[i].x, b[i].x, a[i].y, b[i].y, t[i].x, t[i].y, bf16);
            mma_16816(c, a[i].z, b[i].z, a[i].w, b[i].w, t[i].z, t[i].w, bf16);
        }
    }
}

// The warps' sums, added in warp order; every lane keeps the places its
// fragment has.
__device__ __forceinline__ void add_warps(const float4 (*part)[32], float (&c)[4])
{
    const int lane = int(threadIdx.x) % 32;
    float4 s = part[0][lane];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) {
        const float4 v = part[w][lane];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    c[0] = s.x;
    c[1] = s.y;
    c[2] = s.z;
    c[3] = s.w;
}

__device__ __forceinline__ void put16(void *p, int64_t i, float v, int bf16)
{
    if (bf16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// g, u and h of 8 hidden units.
__global__ void __launch_bounds__(32 * kRowWarps) ffn_rows_up_kernel(const FfnRows a)
{
    __shared__ float4 part[kRowWarps][32];
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32, g = lane / 4;
    const int64_t unit = int64_t(blockIdx.x) * 8 + g;  // hidden is a multiple of 8
    griddep_wait();
    float c[4] = {};
    stream_k(static_cast<const uint16_t *>(a.w_gate) + unit * a.ld_gate,
             static_cast<const uint16_t *>(a.w_up) + unit * a.ld_up,
             g < a.tokens ? static_cast<const uint16_t *>(a.x) + g * a.ldx : nullptr, a.width, a.bf16, c);
    griddep_launch_dependents();  // the next kernel is set up, and waits for this one's end
    part[warp][lane] = make_float4(c[0], c[1], c[2], c[3]);
    __syncthreads();
    if (warp > 0) return;
    float s[4];
    add_warps(part, s);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int token = (lane % 4) * 2 + e;
        if (token >= a.tokens) continue;
        const int64_t i = int64_t(token) * a.hidden + unit;
        float act, slope;
        if (a.act == kSilu)
            activate<kSilu>(s[e], act, slope);
        else if (a.act == kGelu)
            activate<kGelu>(s[e], act, slope);
        else
            activate<kRelu>(s[e], act, slope);
        put16(a.h, i, act * s[2 + e], a.bf16);
        if (a.g) {
            put16(a.g, i, s[e], a.bf16);
            put16(a.u, i, s[2 + e], a.bf16);
        }
    }
}

// y of 16 output features.
__global__ void __launch_bounds__(32 * kRowWarps) ffn_rows_down_kernel(const FfnRows a)
{
    __shared__ float4 part[kRowWarps][32];
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32, g = lane / 4;
    const int64_t lo = int64_t(blockIdx.x) * 16 + g, hi = lo + 8;
    const uint16_t *w = static_cast<const uint16_t *>(a.w_down);
    griddep_wait();
    float c[4] = {};
    stream_k(lo < a.width ? w + lo * a.ld_down : nullptr, hi < a.width ? w + hi * a.ld_down : nullptr,
             g < a.tokens ? static_cast<const uint16_t *>(a.h) + g * a.hidden : nullptr, a.hidden, a.bf16, c);
    griddep_launch_dependents();
    part[warp][lane] = make_float4(c[0], c[1], c[2], c[3]);
    __syncthreads();
    if (warp > 0) return;
    float s[4];
    add_warps(part, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int token = (lane % 4) * 2 + e % 2;
        const int64_t row = e < 2 ? lo : hi;
        if (token < a.tokens && row < a.width) put16(a.y, int64_t(token) * a.ldy + row, s[e], a.bf16);
    }
}

int ffn_rows_forward(const FfnRows &a, cudaStream_t s)
{
    const int rc = launch(ffn_rows_up_kernel, dim3(unsigned(a.hidden / 8)), dim3(32 * kRowWarps), 0, s, 1, a);
    if (rc != kOk) return rc;
    return launch(ffn_rows_down_kernel, dim3(unsigned((a.width + 15) / 16)), dim3(32 * kRowWarps), 0, s, 1, a);
}

}  // namespace tg
