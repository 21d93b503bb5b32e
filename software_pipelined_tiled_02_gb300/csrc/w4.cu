// w4.cu -- products of a few rows with matrices of 4-bit weights, and their C ABI.
//
//   y[t][n] = sum over k of x[t][k] w[n][k],   w[n][k] = (q[n][k] - z[n][k / G]) s[n][k / G]
//
// with q and z between 0 and 15, one scale s and one zero point z for every G
// weights of a row.  With an expert for each pair of a token and a choice, every
// pair has the matrix that its expert names.
//
// A warp's m16n8k16 steps take 16 weight rows and 8 tokens.  q - z is a whole
// number of at most 15, exact in fp16 and bf16, so the tensor core sums exact
// products of a group in fp32, and the group's scale multiplies that sum in fp32:
// no rounding but the sums' and the output's.
//   A nibble becomes a number by its bits alone: or-ed into the mantissa of 1024
// (fp16) or 128 (bf16), from which 1024 + z or 128 + z is subtracted, two at a
// time.  A word's nibbles come out as the pairs (0, 4), (1, 5), (2, 6), (3, 7);
// the order of k does not matter to a sum as long as x is taken in the same one,
// so x's pairs are permuted, not the weights.
//
// What bounds it: the weights' bytes.  The warps of a CTA share out k, each with
// several 16-byte loads a lane on their way, and add their sums in warp order.

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"
#include "tgemm.h"

namespace tg {

constexpr int kW4Warps = 8;

struct W4 {
    const uint16_t *x;
    int64_t ldx;
    const uint8_t *packed;
    const void *scales;
    const uint8_t *zeros;   // NULL: 8
    const int *experts;     // NULL: one matrix
    void *y;
    int64_t n, k, groups;   // groups of a row
    int64_t group;
    int pairs;              // rows of y
    int each;               // rows of y for one row of x
    int num_experts;
    bool scales_f32, y_f32;
};

// VW words of 8 weights, which are not read again: kept out of L1.
template <int VW>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[VW])
{
    if constexpr (VW == 4)
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(p));
    else if constexpr (VW == 2)
        asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
}

template <bool BF16>
__device__ __forceinline__ void mma_w4(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1)
{
    if constexpr (BF16)
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

// 8 nibbles as four pairs of q - z; `base` holds 1024 + z or 128 + z twice.
template <bool BF16>
__device__ __forceinline__ void spread(uint32_t w, uint32_t base, uint32_t (&a)[4])
{
    constexpr uint32_t one = BF16 ? 0x43004300u : 0x64006400u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | one;
        if constexpr (BF16) {
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&base));
            a[i] = *reinterpret_cast<const uint32_t *>(&d);
        } else {
            const __half2 d =
                __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&base));
            a[i] = *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ float scale_at(const W4 &p, int64_t i)
{
    if (p.scales_f32) return static_cast<const float *>(p.scales)[i];
    if constexpr (BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.scales)[i]);
    else
        return __half2float(static_cast<const __half *>(p.scales)[i]);
}

// Pairs that take expert `e` (-1: none that exists), from pair `from` on, in
// order, at most `most`; the place to go on from.  One warp.
__device__ __forceinline__ int list_pairs(const W4 &p, int e, int from, int most, int *list, int &count)
{
    const int lane = int(threadIdx.x) % 32;
    count = 0;
    while (from < p.pairs && count < most) {
        int v = -2;
        if (from + lane < p.pairs) {
            v = p.experts[from + lane];
            if (v < 0 || v >= p.num_experts) v = -1;
        }
        const unsigned found = __ballot_sync(0xffffffffu, v == e);
        const int place = count + __popc(found & ((1u << lane) - 1u));
        if (v == e && place < most) list[place] = from + lane;
        const int taken = min(most - count, __popc(found));
        if (count + __popc(found) > most) {  // go on behind the last one taken
            const unsigned last = __ballot_sync(0xffffffffu, v == e && place == most - 1);
            from += __ffs(int(last));
        } else {
            from += 32;
        }
        count += taken;
    }
    return min(from, p.pairs);
}

// 16 R weight rows, up to 8 NT tokens at a time.  Chunks of 32 VW weights of a
// row, 16 or 8 or 4 bytes a lane: a chunk lies in one group.
template <bool BF16, int VW, int R, int NT>
__global__ void __launch_bounds__(32 * kW4Warps) w4_kernel(const W4 p)
{
    constexpr int kChunkK = 32 * VW;
    constexpr int kAhead = R == 1 ? 4 : 2;  // chunks whose weights are on their way
    __shared__ float part[kW4Warps][R * 16][8 * NT + 1];
    __shared__ int list[8 * NT], listed[2];
    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32, g = lane / 4, c = lane % 4;
    const int64_t row0 = int64_t(blockIdx.x) * (16 * R);
    griddep_wait();
    griddep_launch_dependents();

    int expert = 0, from = int(blockIdx.z) * 8 * NT;
    if (p.experts) {
        // Slot y is pair y's expert if no pair before names it, or with more pairs
        // than experts expert y itself.
        expert = int(blockIdx.y);
        if (p.pairs <= p.num_experts) {
            const int v = p.experts[blockIdx.y];
            expert = v < 0 || v >= p.num_experts ? -1 : v;
            bool before = false;
            for (int i = int(threadIdx.x); i < int(blockIdx.y); i += 32 * kW4Warps) {
                const int o = p.experts[i];
                before |= (o < 0 || o >= p.num_experts ? -1 : o) == expert;
            }
            if (__syncthreads_or(before)) return;
        } else if (expert == p.num_experts) {
            expert = -1;
        }
        from = 0;
    }
    const uint8_t *packed = p.packed;
    int64_t first_group = 0;
    if (expert > 0) {
        packed += int64_t(expert) * p.n * (p.k / 2);
        first_group = int64_t(expert) * p.n * p.groups;
    }
    const int chunks = int(p.k / kChunkK);

    for (;;) {
        int count;
        if (p.experts) {
            if (warp == 0) {
                int n;
                const int next = list_pairs(p, expert, from, 8 * NT, list, n);
                if (lane == 0) {
                    listed[0] = n;
                    listed[1] = next;
                }
            }
            __syncthreads();
            count = listed[0];
            from = listed[1];
            if (count == 0) return;
        } else {
            count = min(8 * NT, p.pairs - from);
        }
        auto pair_at = [&](int i) { return p.experts ? list[i] : from + i; };
        float total[R][NT][4] = {};
        if (expert >= 0) {
            const uint16_t *xs[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int i = t * 8 + g;
                xs[t] = i < count ? p.x + int64_t(pair_at(i) / p.each) * p.ldx + c * (8 * VW) : nullptr;
            }
            const uint8_t *rows[2 * R];
            int64_t group0[2 * R];
#pragma unroll
            for (int r = 0; r < 2 * R; ++r) {
                const int64_t row = min(row0 + r * 8 + g, p.n - 1);  // past the end: computed and dropped
                rows[r] = packed + row * (p.k / 2) + c * (4 * VW);
                group0[r] = first_group + row * p.groups;
            }
            for (int ch0 = warp; ch0 < chunks; ch0 += kW4Warps * kAhead) {
                uint32_t w[kAhead][2 * R][VW];
                float sc[kAhead][2 * R];
                uint32_t base[kAhead][2 * R];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int ch = min(ch0 + a * kW4Warps, chunks - 1);
                    const int64_t group = int64_t(ch) * kChunkK / p.group;
#pragma unroll
                    for (int r = 0; r < 2 * R; ++r) {
                        load_words<VW>(rows[r] + int64_t(ch) * (kChunkK / 2), w[a][r]);
                        sc[a][r] = scale_at<BF16>(p, group0[r] + group);
                        const uint32_t z = p.zeros ? p.zeros[group0[r] + group] & 15u : 8u;
                        base[a][r] = (BF16 ? 0x43004300u : 0x64006400u) + z * 0x00010001u;
                    }
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int ch = ch0 + a * kW4Warps;
                    if (ch >= chunks) break;
                    float acc[R][NT][4] = {};
#pragma unroll
                    for (int v = 0; v < VW; ++v) {
                        uint32_t b[NT][4];
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            uint4 q = make_uint4(0u, 0u, 0u, 0u);
                            if (xs[t]) q = *reinterpret_cast<const uint4 *>(xs[t] + int64_t(ch) * kChunkK + v * 8);
                            b[t][0] = __byte_perm(q.x, q.z, 0x5410);
                            b[t][1] = __byte_perm(q.x, q.z, 0x7632);
                            b[t][2] = __byte_perm(q.y, q.w, 0x5410);
                            b[t][3] = __byte_perm(q.y, q.w, 0x7632);
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            uint32_t lo[4], hi[4];
                            spread<BF16>(w[a][2 * r][v], base[a][2 * r], lo);
                            spread<BF16>(w[a][2 * r + 1][v], base[a][2 * r + 1], hi);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                mma_w4<BF16>(acc[r][t], lo[0], hi[0], lo[1], hi[1], b[t][0], b[t][1]);
                                mma_w4<BF16>(acc[r][t], lo[2], hi[2], lo[3], hi[3], b[t][2], b[t][3]);
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                total[r][t][e] = fmaf(acc[r][t][e], sc[a][2 * r + e / 2], total[r][t][e]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[warp][r * 16 + e / 2 * 8 + g][t * 8 + c * 2 + e % 2] = total[r][t][e];
        __syncthreads();
        for (int i = int(threadIdx.x); i < R * 16 * count; i += 32 * kW4Warps) {
            const int row = i % (R * 16), t = i / (R * 16);
            if (row0 + row >= p.n) continue;
            float v = part[0][row][t];
#pragma unroll
            for (int w = 1; w < kW4Warps; ++w) v += part[w][row][t];
            const int64_t at = int64_t(pair_at(t)) * p.n + row0 + row;
            if (p.y_f32)
                static_cast<float *>(p.y)[at] = v;
            else if (BF16)
                static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
            else
                static_cast<__half *>(p.y)[at] = __float2half_rn(v);
        }
        if (!p.experts || from >= p.pairs) return;
        __syncthreads();  // `part` and the list are read
    }
}

template <bool BF16, int VW, int R, int NT>
static int w4_launch(const W4 &p, cudaStream_t s)
{
    const int64_t blocks = (p.n + 16 * R - 1) / (16 * R);
    const int slots = !p.experts ? 1 : p.pairs <= p.num_experts ? p.pairs : p.num_experts + 1;
    const int passes = p.experts ? 1 : (p.pairs + 8 * NT - 1) / (8 * NT);
    if (blocks > 2147483647 || slots > 65535 || passes > 65535) return kErrInvalidArg;
    return launch(w4_kernel<BF16, VW, R, NT>, dim3(unsigned(blocks), unsigned(slots), unsigned(passes)),
                  dim3(32 * kW4Warps), 0, s, 1, p);
}

template <bool BF16, int VW>
static int w4_shape(const W4 &p, cudaStream_t s)
{
    // tokens that one matrix can have
    const int tokens = p.experts ? (p.pairs + p.num_experts - 1) / p.num_experts : p.pairs;
    if (tokens <= 8) return w4_launch<BF16, VW, 1, 1>(p, s);
    if (tokens <= 16) return w4_launch<BF16, VW, 2, 2>(p, s);
    return w4_launch<BF16, VW, 2, 4>(p, s);
}

template <bool BF16>
static int w4(const W4 &p, cudaStream_t s)
{
    if (p.group % 128 == 0) return w4_shape<BF16, 4>(p, s);
    if (p.group % 64 == 0) return w4_shape<BF16, 2>(p, s);
    return w4_shape<BF16, 1>(p, s);
}

}  // namespace tg

using namespace tg;

extern "C" int tgemm_gemm_fourbit(int64_t pairs, int64_t n, int64_t k, int64_t group, int dtype, const void *x, int64_t ldx,
                             int64_t each, const uint8_t *packed, const void *scales, int scale_dtype,
                             const uint8_t *zeros, const int *experts, int64_t num_experts, void *y, int y_dtype,
                             tgemm_stream_t stream)
{
    if ((dtype != kF16 && dtype != kBF16) || (scale_dtype != dtype && scale_dtype != kF32) ||
        (y_dtype != dtype && y_dtype != kF32))
        return kErrUnsupportedDtype;
    if (pairs < 0 || pairs > (1 << 20) || n < 1 || n > (1 << 28) || k < 1 || k > (1 << 28) || each < 1 || pairs % each)
        return kErrInvalidArg;
    if (group < 32 || group % 32 || k % group) return kErrInvalidArg;
    if (num_experts < 1 || num_experts > 65534 || (!experts && num_experts != 1)) return kErrInvalidArg;
    Device d;
    const int rc = current_device(d);
    if (rc != kOk) return rc;
    if (!d.gb300) return kErrArch;
    if (pairs == 0) return kOk;
    if (!x || !packed || !scales || !y || (pairs > each && ldx < k)) return kErrInvalidArg;
    if (!aligned16(x) || ldx % 8 || !aligned16(packed) || reinterpret_cast<uintptr_t>(scales) % dtype_bytes(scale_dtype) ||
        reinterpret_cast<uintptr_t>(y) % dtype_bytes(y_dtype) || reinterpret_cast<uintptr_t>(experts) % 4)
        return kErrAlignment;
    W4 p{};
    p.x = static_cast<const uint16_t *>(x);
    p.ldx = ldx;
    p.packed = packed;
    p.scales = scales;
    p.zeros = zeros;
    p.experts = experts;
    p.y = y;
    p.n = n;
    p.k = k;
    p.group = group;
    p.groups = k / group;
    p.pairs = int(pairs);
    p.each = int(each);
    p.num_experts = int(num_experts);
    p.scales_f32 = scale_dtype == kF32;
    p.y_f32 = y_dtype == kF32;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == kBF16 ? w4<true>(p, s) : w4<false>(p, s);
}
