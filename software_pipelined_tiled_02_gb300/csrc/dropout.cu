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
// HBM-bound: each tensor is read or written once.

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
    uint64_t threshold;  // 0 .. 2^32: an element is kept when its word is not below it
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

// Vectors of V elements (V a multiple of 4, so whole blocks), grid-stride; the
// last n % V elements one by one.  V = 1: every element by itself, for
// pointers off the 16-byte boundary.
template <class T, int V>
__global__ void __launch_bounds__(256) dropout_kernel(const Dropout a)
{
    griddep_wait();
    griddep_launch_dependents();
    const T *x = static_cast<const T *>(a.x);
    const T *res = static_cast<const T *>(a.residual);
    T *y = static_cast<T *>(a.y);
    const int64_t stride = int64_t(gridDim.x) * 256, first = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t nvec = a.n / V;
    for (int64_t i = first; i < nvec; i += stride) {
        const Pack<T, V> q = load_pack<T, V>(x + i * V);
        Pack<T, V> b, o;
        if (res) b = load_pack<T, V>(res + i * V);
#pragma unroll
        for (int e0 = 0; e0 < V; e0 += 4) {
            uint32_t c[4];
            philox(uint64_t(i * V + e0) / 4, a, c);
#pragma unroll
            for (int e = e0; e < e0 + 4 && e < V; ++e) {
                const uint32_t word = V == 1 ? word_of(c, i) : c[e & 3];
                float z = word >= a.threshold ? to_f32(q.v[e]) * a.scale : 0.f;
                if (res) z += to_f32(b.v[e]);
                o.v[e] = from_f32<T>(z);
            }
        }
        store_pack<T, V>(y + i * V, o);
    }
    if (V > 1) {
        const int64_t i = nvec * V + first;  // fewer than V elements are left: one per thread
        if (i < a.n) {
            uint32_t c[4];
            philox(uint64_t(i) / 4, a, c);
            float z = word_of(c, i) >= a.threshold ? to_f32(x[i]) * a.scale : 0.f;
            if (res) z += to_f32(res[i]);
            y[i] = from_f32<T>(z);
        }
    }
}

template <class T>
static int dropout(const Dropout &a, bool vec, int sms, cudaStream_t s)
{
    constexpr int V = 16 / int(sizeof(T));
    const int64_t work = vec ? a.n / V + 1 : a.n;
    const int64_t blocks = (work + 255) / 256, cap = int64_t(8) * sms;
    const dim3 grid(unsigned(blocks < cap ? blocks : cap));
    return vec ? launch(dropout_kernel<T, V>, grid, dim3(256), 0, s, 1, a)
               : launch(dropout_kernel<T, 1>, grid, dim3(256), 0, s, 1, a);
}

}  // namespace tg

using namespace tg;

extern "C" int tgemm_dropout(int64_t n, int dtype, const void *x, const void *residual, void *y, double p,
                             uint64_t seed, uint64_t offset, tgemm_stream_t stream)
{
    if (dtype != kF16 && dtype != kBF16 && dtype != kF32) return kErrUnsupportedDtype;
    if (n < 0 || n > (int64_t(1) << 60) || !(p >= 0.0 && p <= 1.0)) return kErrInvalidArg;
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
    a.threshold = uint64_t(std::nearbyint(p * 4294967296.0));
    a.scale = p < 1.0 ? float(1.0 / (1.0 - p)) : 0.f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = at % 16 == 0;
    if (dtype == kF32) return dropout<float>(a, vec, d.sms, s);
    return dtype == kF16 ? dropout<__half>(a, vec, d.sms, s) : dropout<__nv_bfloat16>(a, vec, d.sms, s);
}
