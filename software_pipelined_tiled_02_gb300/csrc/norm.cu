// norm.cu -- layer normalisation over the rows of a matrix, forward and
// backward, for GB300 (sm_103a), and its C ABI.
//
// Forward.  mean = sum x / D, var = sum (x - mean)^2 / D, r = 1/sqrt(var + eps),
// y = (x - mean) r w + b.  A row stays in the registers of its warp or CTA
// between the two sums and the output, so it is read once.
//
// Backward, with xh = (x - mean) r and q = dy w:
//   dx = r (q - mean(q) - xh mean(q xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
// Each CTA walks over rows and keeps its columns' sums of dy xh and dy in
// registers; it writes them once, and a second kernel adds the CTAs' sums in
// a fixed order, so results do not depend on timing.
//
// All sums and statistics are fp32; outputs are rounded once.  Both passes are
// bound by HBM: 2 (forward) and 3 (backward) row-sized transfers.

#include <cuda_runtime.h>

#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"
#include "tgemm.h"

namespace tg {

struct NormFwd {
    int64_t rows, width, ldx, ldy;
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    float eps, inv_width;
    bool w_f32;
};

struct NormBwd {
    int64_t rows, width, lddy, ldx, lddx;
    const void *dy, *x, *w;
    const float *mean, *rstd;
    void *dx;
    float *part;  // [2][parts][width]: sums of dy xh, then of dy
    int parts;
    float inv_width;
    bool w_f32;
};

// Sum of one value over the warps of a CTA (every thread gets it); `buf` holds
// one float per warp and is used once between two barriers.
__device__ __forceinline__ float cta_sum(float v, float *buf)
{
    v = warp_sum(v);
    const int warps = int(blockDim.x) / 32;
    if ((threadIdx.x & 31u) == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += buf[i];
    return s;
}

// One row per warp (CTA false) or per CTA; thread t holds the row's vectors
// t, t + threads, ...: NV of them.
template <class T, int V, int NV, bool CTA>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormFwd a)
{
    __shared__ float buf[2][32];
    const int threads = CTA ? int(blockDim.x) : 32;
    const int t = CTA ? int(threadIdx.x) : int(threadIdx.x) % 32;
    const int64_t row = CTA ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    griddep_wait();
    griddep_launch_dependents();
    if (row >= a.rows) return;  // whole warps; a CTA's row is always inside
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const int nvec = int(a.width / V);
    Pack<T, V> q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (t + j * threads < nvec) q[j] = load_pack<T, V>(x + int64_t(t + j * threads) * V);
    float v[NV][V], s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const bool in = t + j * threads < nvec;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[j][e] = in ? to_f32(q[j].v[e]) : 0.f;
            s += v[j][e];
        }
    }
    const float mean = (CTA ? cta_sum(s, buf[0]) : warp_sum(s)) * a.inv_width;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (t + j * threads < nvec) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[j][e] -= mean;
                ss += v[j][e] * v[j][e];
            }
        }
    }
    const float var = (CTA ? cta_sum(ss, buf[1]) : warp_sum(ss)) * a.inv_width;
    const float r = 1.f / sqrtf(var + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = r;
    }
    T *y = static_cast<T *>(a.y) + row * a.ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = t + j * threads;
        if (i >= nvec) continue;
        float w[V], b[V];
        if (a.w) load_weights<T, V>(a.w, int64_t(i) * V, a.w_f32, w);
        if (a.b) load_weights<T, V>(a.b, int64_t(i) * V, a.w_f32, b);
        Pack<T, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float z = v[j][e] * r;
            if (a.w) z *= w[e];
            if (a.b) z += b[e];
            o.v[e] = from_f32<T>(z);
        }
        store_pack<T, V>(y + int64_t(i) * V, o);
    }
}

// Rows too wide for the registers of a CTA: three passes over the row, the
// later ones from L2.
template <class T>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const NormFwd a)
{
    __shared__ float buf[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    T *y = static_cast<T *>(a.y) + row * a.ldy;
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x) s += to_f32(x[i]);
    const float mean = cta_sum(s, buf[0]) * a.inv_width;
    float ss = 0.f;
    for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x) {
        const float d = to_f32(x[i]) - mean;
        ss += d * d;
    }
    const float r = 1.f / sqrtf(cta_sum(ss, buf[1]) * a.inv_width + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = r;
    }
    for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x) {
        float z = (to_f32(x[i]) - mean) * r, w[1], b[1];
        if (a.w) {
            load_weights<T, 1>(a.w, i, a.w_f32, w);
            z *= w[0];
        }
        if (a.b) {
            load_weights<T, 1>(a.b, i, a.w_f32, b);
            z += b[0];
        }
        y[i] = from_f32<T>(z);
    }
}

// Sums of two values over the `warps` warps of a group, which meet on hardware
// barrier `bar`; `buf` holds two floats per warp of the group.  Rows alternate
// between two buffers, so one barrier per row is enough: a warp writes buffer
// k again two rows later, after every warp of the group has passed the barrier
// of the row between, which each reaches only once it has read buffer k.
__device__ __forceinline__ void group_sum2(float &x, float &y, float *buf, int warps, int w, int bar)
{
    x = warp_sum(x);
    y = warp_sum(y);
    if (warps == 1) return;
    if ((threadIdx.x & 31u) == 0) {
        buf[2 * w] = x;
        buf[2 * w + 1] = y;
    }
    named_bar_sync(uint32_t(bar), uint32_t(warps) * 32u);
    x = y = 0.f;
    for (int i = 0; i < warps; ++i) {
        x += buf[2 * i];
        y += buf[2 * i + 1];
    }
}

constexpr int kNormBwdThreads = 512;

// Groups of `warps` warps take rows round robin over the whole grid; thread t
// of a group holds the row's vectors t, t + 32 warps, ...: NV of them, and the
// same columns' running sums of dy xh and dy.  At the end the CTA's groups add
// their sums in shared memory in group order, and the CTA writes one partial
// row of each.
template <class T, int V, int NV>
__global__ void __launch_bounds__(kNormBwdThreads) norm_bwd_kernel(const NormBwd a, int warps)
{
    __shared__ float buf[2][2 * kNormBwdThreads / 32];
    extern __shared__ float sums[];  // [2][width], with more than one group
    const int groups = kNormBwdThreads / 32 / warps;
    const int g = int(threadIdx.x) / 32 / warps, gw = int(threadIdx.x) / 32 - g * warps;
    const int threads = warps * 32;
    const int t = int(threadIdx.x) - g * threads;
    const int nvec = int(a.width / V);
    griddep_wait();
    griddep_launch_dependents();
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[j][e] = 1.f;
            dw[j][e] = db[j][e] = 0.f;
        }
        if (a.w && t + j * threads < nvec) load_weights<T, V>(a.w, int64_t(t + j * threads) * V, a.w_f32, w[j]);
    }
    int k = 0;
    for (int64_t row = int64_t(blockIdx.x) * groups + g; row < a.rows; row += int64_t(gridDim.x) * groups) {
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
        Pack<T, V> qx[NV], qd[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (t + j * threads < nvec) {
                qx[j] = load_pack<T, V>(x + int64_t(t + j * threads) * V);
                qd[j] = load_pack<T, V>(dy + int64_t(t + j * threads) * V);
            }
        }
        const float mean = a.mean[row], r = a.rstd[row];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (t + j * threads < nvec) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (to_f32(qx[j].v[e]) - mean) * r, d = to_f32(qd[j].v[e]);
                    const float q = d * w[j][e];
                    s1 += q;
                    s2 += q * xh;
                    dw[j][e] += d * xh;
                    db[j][e] += d;
                }
            }
        }
        group_sum2(s1, s2, buf[k] + 2 * g * warps, warps, gw, 1 + g);
        k ^= 1;
        s1 *= a.inv_width;
        s2 *= a.inv_width;
        T *dx = static_cast<T *>(a.dx) + row * a.lddx;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (t + j * threads >= nvec) continue;
            Pack<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xh = (to_f32(qx[j].v[e]) - mean) * r, q = to_f32(qd[j].v[e]) * w[j][e];
                o.v[e] = from_f32<T>(r * (q - s1 - xh * s2));
            }
            store_pack<T, V>(dx + int64_t(t + j * threads) * V, o);
        }
    }
    if (!a.part) return;
    float *pw = a.part + int64_t(blockIdx.x) * a.width, *pb = pw + int64_t(a.parts) * a.width;
    float *sw = groups > 1 ? sums : pw, *sb = groups > 1 ? sums + a.width : pb;
    for (int i = 0; i < groups; ++i) {
        if (g == i) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (t + j * threads) * V;
                if (t + j * threads >= nvec) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sw[c + e] = i ? sw[c + e] + dw[j][e] : dw[j][e];
                    sb[c + e] = i ? sb[c + e] + db[j][e] : db[j][e];
                }
            }
        }
        if (groups > 1) __syncthreads();
    }
    if (groups > 1) {
        for (int c = int(threadIdx.x); c < a.width; c += kNormBwdThreads) {
            pw[c] = sw[c];
            pb[c] = sb[c];
        }
    }
}

// Rows too wide for a CTA's registers: the row's sums, then dx, from L2.  The
// column sums of such matrices come from norm_bwd_cols_kernel.
template <class T>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const NormBwd a)
{
    __shared__ float buf[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
    T *dx = static_cast<T *>(a.dx) + row * a.lddx;
    const float mean = a.mean[row], r = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x) {
        float w[1] = {1.f};
        if (a.w) load_weights<T, 1>(a.w, i, a.w_f32, w);
        const float q = to_f32(dy[i]) * w[0];
        s1 += q;
        s2 += q * ((to_f32(x[i]) - mean) * r);
    }
    s1 = cta_sum(s1, buf[0]) * a.inv_width;
    s2 = cta_sum(s2, buf[1]) * a.inv_width;
    for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x) {
        float w[1] = {1.f};
        if (a.w) load_weights<T, 1>(a.w, i, a.w_f32, w);
        const float q = to_f32(dy[i]) * w[0], xh = (to_f32(x[i]) - mean) * r;
        dx[i] = from_f32<T>(r * (q - s1 - xh * s2));
    }
}

// Partial column sums: CTA (x, y) takes 256 columns and rows y, y + parts, ...
template <class T>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(const NormBwd a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (c >= a.width) return;
    float dw = 0.f, db = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += a.parts) {
        const float d = to_f32(static_cast<const T *>(a.dy)[row * a.lddy + c]);
        const float v = to_f32(static_cast<const T *>(a.x)[row * a.ldx + c]);
        dw += d * ((v - a.mean[row]) * a.rstd[row]);
        db += d;
    }
    a.part[int64_t(blockIdx.y) * a.width + c] = dw;
    a.part[(int64_t(a.parts) + blockIdx.y) * a.width + c] = db;
}

// Adds the partial rows of dw (blockIdx.y 0) and db (1): 32 columns a CTA, its
// warps take parts w, w + 8, ... and are added in warp order.
template <class W>
__global__ void __launch_bounds__(256) norm_bwd_reduce_kernel(const float *part, int parts, int64_t width, W *dw, W *db)
{
    __shared__ float s[8][32];
    griddep_wait();
    griddep_launch_dependents();
    W *out = blockIdx.y ? db : dw;
    if (!out) return;
    const float *p = part + int64_t(blockIdx.y) * parts * width;
    const int lane = int(threadIdx.x) % 32, w = int(threadIdx.x) / 32;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float v = 0.f;
    if (c < width)
        for (int i = w; i < parts; i += 8) v += p[int64_t(i) * width + c];
    s[w][lane] = v;
    __syncthreads();
    if (w == 0 && c < width) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][lane];
        out[c] = from_f32<W>(v);
    }
}

// ---------------------------------------------------------------- host side

// Threads per row: the fewest warps (a power of two) whose threads hold the
// row in at most `most` vectors each, up to `max_warps`; false if the row does
// not fit.
static bool row_shape(int64_t nvec, int most, int last, int max_warps, int *warps, int *nv)
{
    int w = 1;
    while (w < max_warps && nvec > int64_t(32) * w * most) w *= 2;
    int n = 1;
    while (n < last && nvec > int64_t(32) * w * n) n *= 2;
    *warps = w;
    *nv = n;
    return nvec <= int64_t(32) * w * n;
}

template <class T, int V, int NV>
static int fwd_launch(const NormFwd &a, int warps, cudaStream_t s)
{
    if (warps == 1) {
        const int per_cta = 4;
        return launch(norm_fwd_kernel<T, V, NV, false>, dim3(unsigned((a.rows + per_cta - 1) / per_cta)),
                      dim3(32 * per_cta), 0, s, 1, a);
    }
    return launch(norm_fwd_kernel<T, V, NV, true>, dim3(unsigned(a.rows)), dim3(unsigned(32 * warps)), 0, s, 1, a);
}

template <class T>
static int fwd(const NormFwd &a, bool vec, cudaStream_t s)
{
    constexpr int V = 16 / int(sizeof(T));
    int warps = 0, nv = 0;
    if (vec && row_shape(a.width / V, 4, 8, 32, &warps, &nv)) {
        switch (nv) {
        case 1: return fwd_launch<T, V, 1>(a, warps, s);
        case 2: return fwd_launch<T, V, 2>(a, warps, s);
        case 4: return fwd_launch<T, V, 4>(a, warps, s);
        default: return fwd_launch<T, V, 8>(a, warps, s);
        }
    }
    if (row_shape(a.width, 16, 16, 32, &warps, &nv)) {
        switch (nv) {
        case 1: return fwd_launch<T, 1, 1>(a, warps, s);
        case 2: return fwd_launch<T, 1, 2>(a, warps, s);
        case 4: return fwd_launch<T, 1, 4>(a, warps, s);
        case 8: return fwd_launch<T, 1, 8>(a, warps, s);
        default: return fwd_launch<T, 1, 16>(a, warps, s);
        }
    }
    return launch(norm_fwd_wide_kernel<T>, dim3(unsigned(a.rows)), dim3(1024), 0, s, 1, a);
}

// CTAs (and partial rows) of the backward pass: one per SM, fewer for few rows.
static int bwd_parts(int64_t rows, int sms) { return rows < 1 ? 1 : rows < sms ? int(rows) : sms; }

template <class T, int V, int NV>
static int bwd_launch(const NormBwd &a, int warps, cudaStream_t s)
{
    const int groups = kNormBwdThreads / 32 / warps;
    const size_t smem = groups > 1 && a.part ? size_t(a.width) * 2 * sizeof(float) : 0;
    return launch(norm_bwd_kernel<T, V, NV>, dim3(unsigned(a.parts)), dim3(kNormBwdThreads), smem, s, 1, a, warps);
}

template <class T>
static int bwd(const NormBwd &a, bool vec, cudaStream_t s)
{
    constexpr int V = 16 / int(sizeof(T));
    constexpr int kMax = kNormBwdThreads / 32;
    int warps = 0, nv = 0;
    if (vec && row_shape(a.width / V, 16 / V, 16 / V, kMax, &warps, &nv)) {
        if (nv == 1) return bwd_launch<T, V, 1>(a, warps, s);
        if (nv == 2) return bwd_launch<T, V, 2>(a, warps, s);
        if constexpr (V == 4) return bwd_launch<T, V, 4>(a, warps, s);
    }
    if (row_shape(a.width, 16, 16, kMax, &warps, &nv)) {
        switch (nv) {
        case 1: return bwd_launch<T, 1, 1>(a, warps, s);
        case 2: return bwd_launch<T, 1, 2>(a, warps, s);
        case 4: return bwd_launch<T, 1, 4>(a, warps, s);
        case 8: return bwd_launch<T, 1, 8>(a, warps, s);
        default: return bwd_launch<T, 1, 16>(a, warps, s);
        }
    }
    int rc = launch(norm_bwd_wide_kernel<T>, dim3(unsigned(a.rows)), dim3(1024), 0, s, 1, a);
    if (rc == kOk && a.part)
        rc = launch(norm_bwd_cols_kernel<T>, dim3(unsigned((a.width + 255) / 256), unsigned(a.parts)), dim3(256), 0, s,
                    1, a);
    return rc;
}

template <class W>
static int reduce(const NormBwd &a, void *dw, void *db, cudaStream_t s)
{
    return launch(norm_bwd_reduce_kernel<W>, dim3(unsigned((a.width + 31) / 32), 2), dim3(256), 0, s, 1,
                  static_cast<const float *>(a.part), a.parts, a.width, static_cast<W *>(dw), static_cast<W *>(db));
}

// Row-wise operators take sizes up to these: a row index fits a grid, a column
// index an int.
constexpr int64_t kMaxRows = 2147483647, kMaxWidth = int64_t(1) << 30;

static int check_norm(int64_t rows, int64_t width, int dtype, int weight_dtype)
{
    if (dtype != kF16 && dtype != kBF16 && dtype != kF32) return kErrUnsupportedDtype;
    if (weight_dtype != dtype && weight_dtype != kF32) return kErrUnsupportedDtype;
    if (rows < 0 || rows > kMaxRows || width < 1 || width > kMaxWidth) return kErrInvalidArg;
    return kOk;
}

static bool aligned_to(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % unsigned(bytes) == 0; }

}  // namespace tg

using namespace tg;

extern "C" {

int tgemm_layer_norm(int64_t rows, int64_t width, int dtype, int weight_dtype, const void *x, int64_t ldx,
                     const void *weight, const void *bias, float eps, void *y, int64_t ldy, float *mean, float *rstd,
                     tgemm_stream_t stream)
{
    int rc = check_norm(rows, width, dtype, weight_dtype);
    if (rc != kOk) return rc;
    if (ldx < width || ldy < width || !(eps >= 0.f)) return kErrInvalidArg;
    Device d;
    if ((rc = current_device(d)) != kOk) return rc;
    if (!d.gb300) return kErrArch;
    if (rows == 0) return kOk;
    if (!x || !y) return kErrInvalidArg;
    const int e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, we) || !aligned_to(bias, we) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return kErrAlignment;
    const bool vec = aligned16(x) && aligned16(y) && aligned16(weight) && aligned16(bias) && ldx * e % 16 == 0 &&
                     ldy * e % 16 == 0 && width * e % 16 == 0;
    const NormFwd a{rows, width, ldx, ldy, x, weight, bias, y, mean, rstd, eps, float(1.0 / double(width)),
                    weight_dtype == kF32};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == kF32) return fwd<float>(a, vec, s);
    return dtype == kF16 ? fwd<__half>(a, vec, s) : fwd<__nv_bfloat16>(a, vec, s);
}

int64_t tgemm_layer_norm_workspace(int64_t rows, int64_t width)
{
    if (rows < 0 || rows > kMaxRows || width < 1 || width > kMaxWidth) return -kErrInvalidArg;
    Device d;
    const int rc = current_device(d);
    if (rc != kOk) return -rc;
    return int64_t(2) * bwd_parts(rows, d.sms) * width * int64_t(sizeof(float));
}

int tgemm_layer_norm_backward(int64_t rows, int64_t width, int dtype, int weight_dtype, const void *dy, int64_t lddy,
                              const void *x, int64_t ldx, const float *mean, const float *rstd, const void *weight,
                              void *dx, int64_t lddx, void *dweight, void *dbias, void *workspace,
                              int64_t workspace_bytes, tgemm_stream_t stream)
{
    int rc = check_norm(rows, width, dtype, weight_dtype);
    if (rc != kOk) return rc;
    if (lddy < width || ldx < width || lddx < width) return kErrInvalidArg;
    Device d;
    if ((rc = current_device(d)) != kOk) return rc;
    if (!d.gb300) return kErrArch;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return kErrInvalidArg;
    const bool sums = dweight || dbias;
    const int e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
    if (!aligned_to(dy, e) || !aligned_to(x, e) || !aligned_to(dx, e) || !aligned_to(weight, we) ||
        !aligned_to(dweight, we) || !aligned_to(dbias, we) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return kErrAlignment;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {  // empty sums
        if ((dweight && cudaMemsetAsync(dweight, 0, size_t(width) * we, s) != cudaSuccess) ||
            (dbias && cudaMemsetAsync(dbias, 0, size_t(width) * we, s) != cudaSuccess)) {
            cudaGetLastError();
            return kErrCuda;
        }
        return kOk;
    }
    const int parts = bwd_parts(rows, d.sms);
    if (sums) {
        if (!workspace || workspace_bytes < int64_t(2) * parts * width * int64_t(sizeof(float))) return kErrInvalidArg;
        if (!aligned16(workspace)) return kErrAlignment;
    }
    const bool vec = aligned16(dy) && aligned16(x) && aligned16(dx) && aligned16(weight) && lddy * e % 16 == 0 &&
                     ldx * e % 16 == 0 && lddx * e % 16 == 0 && width * e % 16 == 0;
    const NormBwd a{rows, width, lddy, ldx, lddx, dy, x, weight, mean, rstd, dx,
                    sums ? static_cast<float *>(workspace) : nullptr, parts, float(1.0 / double(width)),
                    weight_dtype == kF32};
    rc = dtype == kF32 ? bwd<float>(a, vec, s) : dtype == kF16 ? bwd<__half>(a, vec, s) : bwd<__nv_bfloat16>(a, vec, s);
    if (rc != kOk || !sums) return rc;
    if (weight_dtype == kF32) return reduce<float>(a, dweight, dbias, s);
    return weight_dtype == kF16 ? reduce<__half>(a, dweight, dbias, s) : reduce<__nv_bfloat16>(a, dweight, dbias, s);
}

}  // extern "C"
