// dropout.cu -- dropout whose mask is computed, never stored, for GB300
// (sm_103a), and its C ABI.
//
// The mask comes from the counter-based generator Philox4x32 with 10 rounds
// (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3", 2011).  Element i of the tensor takes word i % 4 of the block whose
// counter is (i / 4, offset) and whose key is the seed; it is kept when that
// word is at least round(p 2^32).  So the forward and the backward pass, and
// any launch shape, form the same mask from (seed, offset) alone.
//
//   y_i = kept_i ? x_i / (1 - p) : 0   (+ residual_i)
//
// A dropped value is replaced, not multiplied, so an infinity or NaN in it
// does not come through.  The sum is formed in fp32 and rounded once.
// HBM-bound: each tensor is read or written once.  8192 x 4096 bf16 with a
// residual: 31.6 us, 6.4 TB/s.

#include <cuda_runtime.h>

#include <cmath>

#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"
#include "tgemm.h"

namespace tg {

struct Dropout {
    int64_t n;
    const void *x, *residual;
    void *y;
    uint32_t key0, key1, off0, off1;
    uint32_t threshold;  // an element is kept when its word is not below it
    float scale;
};

// The four words of block `block`.
__device__ __forceinline__ void philox(uint64_t block, const Dropout &a, uint32_t (&c)[4])
{
    c[0] = uint32_t(block);
    c[1] = uint32_t(block >> 32);
    c[2] = a.off0;
    c[3] = a.off1;
    uint32_t k0 = a.key0, k1 = a.key1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = uint64_t(c[0]) * 0xD2511F53u, p1 = uint64_t(c[2]) * 0xCD9E8D57u;
        c[0] = uint32_t(p1 >> 32) ^ c[1] ^ k0;
        c[1] = uint32_t(p1);
        c[2] = uint32_t(p0 >> 32) ^ c[3] ^ k1;
        c[3] = uint32_t(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Word i % 4 of a block.
__device__ __forceinline__ uint32_t word_of(const uint32_t (&c)[4], int64_t i)
{
    return (i & 2) ? ((i & 1) ? c[3] : c[2]) : ((i & 1) ? c[1] : c[0]);
}

// Each thread takes one 16-byte vector (whole blocks of words) of a CTA's 256:
// its loads are on their way while it forms its words, and the 8 CTAs of an SM
// fill in for one another (8192 x 4096 bf16 with residual: 31.5 us, 6.4 TB/s; a
// persistent loop with the next vector's loads ahead took 39 us at the half
// occupancy its registers allowed).  The last CTA also takes the last elements
// one by one.
template <class T, bool RES>
__global__ void __launch_bounds__(256, 8) dropout_kernel(const Dropout a)
{
    constexpr int V = 16 / int(sizeof(T));
    const T *x = static_cast<const T *>(a.x);
    const T *res = static_cast<const T *>(a.residual);
    T *y = static_cast<T *>(a.y);
    const int64_t nvec = a.n / V, at = int64_t(blockIdx.x) * 256 + threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    if (at < nvec) {
        const uint4 q = reinterpret_cast<const uint4 *>(x)[at];
        uint4 b = make_uint4(0u, 0u, 0u, 0u);
        if (RES) b = reinterpret_cast<const uint4 *>(res)[at];
        uint32_t c[V / 4][4];
#pragma unroll
        for (int k = 0; k < V / 4; ++k) philox(uint64_t(at) * (V / 4) + k, a, c[k]);
        F2 v[V / 2], r[V / 2];
        unpack16<T>(q, v);
        if (RES) unpack16<T>(b, r);
        const F2 scale = f2(a.scale);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const F2 none = RES ? r[e] : f2(0.f);
            const float2 kept = split(RES ? fma2(v[e], scale, none) : v[e] * scale), dropped = split(none);
            v[e] = f2(c[e / 2][e % 2 * 2] >= a.threshold ? kept.x : dropped.x,
                      c[e / 2][e % 2 * 2 + 1] >= a.threshold ? kept.y : dropped.y);
        }
        reinterpret_cast<uint4 *>(y)[at] = pack16<T>(v);
    }
    const int64_t i = blockIdx.x + 1 == gridDim.x ? nvec * V + threadIdx.x : a.n;  // fewer than V are left
    if (i < a.n) {
        uint32_t c[4];
        philox(uint64_t(i) / 4, a, c);
        const float none = RES ? to_f32(res[i]) : 0.f;
        y[i] = from_f32<T>(word_of(c, i) >= a.threshold ? fmaf(to_f32(x[i]), a.scale, none) : none);
    }
}

// Every element by itself, for pointers off the 16-byte boundary.
template <class T>
__global__ void __launch_bounds__(256) dropout_single_kernel(const Dropout a)
{
    const T *x = static_cast<const T *>(a.x);
    const T *res = static_cast<const T *>(a.residual);
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < a.n; i += int64_t(gridDim.x) * 256) {
        uint32_t c[4];
        philox(uint64_t(i) / 4, a, c);
        const float none = res ? to_f32(res[i]) : 0.f;
        static_cast<T *>(a.y)[i] =
            from_f32<T>(word_of(c, i) >= a.threshold ? fmaf(to_f32(x[i]), a.scale, none) : none);
    }
}

template <class T>
static int dropout(const Dropout &a, bool vec, int sms, cudaStream_t s)
{
    constexpr int V = 16 / int(sizeof(T));
    const int64_t blocks = ((vec ? a.n / V + 1 : a.n) + 255) / 256, cap = int64_t(8) * sms;
    const dim3 grid(unsigned(vec || blocks < cap ? blocks : cap));
    if (!vec) return launch(dropout_single_kernel<T>, grid, dim3(256), 0, s, 1, a);
    return a.residual ? launch(dropout_kernel<T, true>, grid, dim3(256), 0, s, 1, a)
                      : launch(dropout_kernel<T, false>, grid, dim3(256), 0, s, 1, a);
}

}  // namespace tg

using namespace tg;

extern "C" int tgemm_dropout(int64_t n, int dtype, const void *x, const void *residual, void *y, double p,
                             uint64_t seed, uint64_t offset, tgemm_stream_t stream)
{
    if (dtype != kF16 && dtype != kBF16 && dtype != kF32) return kErrUnsupportedDtype;
    if (n < 0 || n > (int64_t(1) << 40) || !(p >= 0.0 && p <= 1.0)) return kErrInvalidArg;
    Device d;
    const int rc = current_device(d);
    if (rc != kOk) return rc;
    if (!d.gb300) return kErrArch;
    if (n == 0) return kOk;
    if (!x || !y) return kErrInvalidArg;
    const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) |
                         reinterpret_cast<uintptr_t>(residual);
    if (at % unsigned(dtype_bytes(dtype))) return kErrAlignment;
    Dropout a{};
    a.n = n;
    a.x = x;
    a.residual = residual;
    a.y = y;
    a.key0 = uint32_t(seed);
    a.key1 = uint32_t(seed >> 32);
    a.off0 = uint32_t(offset);
    a.off1 = uint32_t(offset >> 32);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const double threshold = std::nearbyint(p * 4294967296.0);
    if (threshold > 4294967295.0) {  // no word reaches 2^32: nothing is kept
        const size_t bytes = size_t(n) * size_t(dtype_bytes(dtype));
        const cudaError_t e = !residual       ? cudaMemsetAsync(y, 0, bytes, s)
                              : residual == y ? cudaSuccess
                                              : cudaMemcpyAsync(y, residual, bytes, cudaMemcpyDeviceToDevice, s);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return kErrCuda;
        }
        return kOk;
    }
    a.threshold = uint32_t(threshold);
    a.scale = float(1.0 / (1.0 - p));
    const bool vec = at % 16 == 0;
    if (dtype == kF32) return dropout<float>(a, vec, d.sms, s);
    return dtype == kF16 ? dropout<__half>(a, vec, d.sms, s) : dropout<__nv_bfloat16>(a, vec, d.sms, s);
}
