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
// All sums and statistics are fp32; outputs are rounded once.  Both passes move
// each tensor once: 2 (forward) and 3 (backward) row-sized transfers.  8192 rows of
// 4096 bf16: forward 26.6 us, 5.0 TB/s; backward 38.2 us with the column sums, 5.3
// TB/s.  Copies of that size reach 5.3 to 6.0 TB/s, dropout with its three tensors
// 6.4; the rest is a step's reductions
// over a row's threads, one after the other.  4000 rows of 3001 fp32, off every
// boundary: backward 35.0 us, 4.1 TB/s.  One row of 4096: 2.6 us.

#include <cuda_runtime.h>

#include <atomic>

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

// One row per warp (CTA false) or per CTA; thread t holds the row's elements
// t, t + threads, ...: NV of them.
template <class T, int NV, bool CTA>
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
    const int width = int(a.width);
    float v[NV], s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = t + j * threads < width ? to_f32(x[t + j * threads]) : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) s += v[j];
    const float mean = (CTA ? cta_sum(s, buf[0]) : warp_sum(s)) * a.inv_width;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (t + j * threads < width) {
            v[j] -= mean;
            ss += v[j] * v[j];
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
        if (i >= width) continue;
        float w[1] = {1.f}, b[1] = {0.f};
        if (a.w) load_weights<T, 1>(a.w, i, a.w_f32, w);
        if (a.b) load_weights<T, 1>(a.b, i, a.w_f32, b);
        y[i] = from_f32<T>(fmaf(v[j] * r, w[0], b[0]));
    }
}

// The same with rows of whole 16-byte vectors: thread t holds vectors t, t +
// threads, ...: NV of them.  Up to 256 threads and 40 registers, so that six
// rows and more share an SM and fill in for one another.
template <class T, int NV, bool CTA, int MAX>
__global__ void __launch_bounds__(MAX, 1536 / MAX) norm_fwd_vec_kernel(const NormFwd a)
{
    constexpr int V = 16 / int(sizeof(T));
    __shared__ float buf[2][32];
    const int threads = CTA ? int(blockDim.x) : 32, warps = threads / 32;
    const int t = CTA ? int(threadIdx.x) : int(threadIdx.x) % 32;
    const int64_t row = CTA ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    auto sum = [&](float v, float *b) {
        v = warp_sum(v);
        if (!CTA) return v;
        if (t % 32 == 0) b[t / 32] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < MAX / 32; ++i)
            if (i < warps) v += b[i];
        return v;
    };
    griddep_wait();
    griddep_launch_dependents();
    if (row >= a.rows) return;  // whole warps; a CTA's row is always inside
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.ldx);
    const int nvec = int(a.width / V);
    uint4 q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (t + j * threads < nvec) q[j] = x[t + j * threads];
    F2 v[NV][V / 2], s = f2(0.f), s_ = f2(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (t + j * threads >= nvec) continue;
        unpack16<T>(q[j], v[j]);
#pragma unroll
        for (int e = 0; e < V / 2; e += 2) {
            s = s + v[j][e];
            s_ = s_ + v[j][e + 1];
        }
    }
    const float mean = sum(sum2(s + s_), buf[0]) * a.inv_width;
    const F2 minus = f2(-mean);
    s = s_ = f2(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (t + j * threads >= nvec) continue;
#pragma unroll
        for (int e = 0; e < V / 2; e += 2) {
            v[j][e] = v[j][e] + minus;
            v[j][e + 1] = v[j][e + 1] + minus;
            s = fma2(v[j][e], v[j][e], s);
            s_ = fma2(v[j][e + 1], v[j][e + 1], s_);
        }
    }
    const float var = sum(sum2(s + s_), buf[1]) * a.inv_width;
    const float r = 1.f / sqrtf(var + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = r;
    }
    const F2 rr = f2(r);
    uint4 *y = reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + row * a.ldy);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = t + j * threads;
        if (i >= nvec) continue;
        float w[V], b[V];
        if (a.w) load_weights<T, V>(a.w, int64_t(i) * V, a.w_f32, w);
        if (a.b) load_weights<T, V>(a.b, int64_t(i) * V, a.w_f32, b);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            F2 z = v[j][e] * rr;
            if (a.w) z = z * f2(w[2 * e], w[2 * e + 1]);
            if (a.b) z = z + f2(b[2 * e], b[2 * e + 1]);
            v[j][e] = z;
        }
        y[i] = pack16<T>(v[j]);
    }
}

// ---------------------------------------------------------------- many rows
//
// Persistent kernels: a CTA's 16 warps form groups of `warps` warps, and the
// groups take rows round robin over the grid.  A row is cut at the 16-byte
// boundaries of memory, not of the row, so that rows of any width (each
// starting `shift` elements past a boundary) move in whole vectors.  A group
// steps over a multiple of 8 rows, so the shift is the same for all its rows,
// thread t always holds the same columns (vectors t, t + 32 warps, ...: NV of
// them), and only the first and the last vector hold foreign elements.

constexpr int kNormThreads = 512;

// This thread's part of its group's rows, and the rows it has in flight: its
// vectors of the next ST rows, copied asynchronously into shared memory that
// no other thread touches, so that a thread waits for its own copies alone.  A
// slot is refilled only after the values read from it have gone through a
// reduction.  EXACT: every row starts on a boundary and is whole vectors wide,
// so no vector holds foreign elements.
template <class T, int NV, int ST, int ARRAYS, bool EXACT>
struct RowRing {
    static constexpr int V = 16 / int(sizeof(T));
    static constexpr uint32_t kBytes = uint32_t(ST) * ARRAYS * NV * kNormThreads * 16;
    uint32_t base;
    int t, threads, shift, width;
    int hop;  // bytes from one of this thread's vectors to the next

    __device__ RowRing(const void *mem, int warps, int width_, int shift_)
        : base(smem_addr(mem) + threadIdx.x * 16), t(int(threadIdx.x) % (warps * 32)), threads(warps * 32),
          shift(EXACT ? 0 : shift_), width(width_), hop(warps * 512)
    {
    }
    // Column of the first element of vector j (negative in a row's first vector).
    __device__ int col(int j) const { return (t + j * threads) * V - shift; }
    __device__ bool some(int j) const { return col(j) < width; }  // holds a column of the row
    __device__ bool whole(int j) const { return EXACT || (col(j) >= 0 && col(j) + V <= width); }  // and nothing else
    __device__ bool valid(int j, int e) const { return EXACT || (col(j) + e >= 0 && col(j) + e < width); }
    __device__ uint32_t at(int slot, int array, int j) const
    {
        return base + uint32_t(slot) * (ARRAYS * NV * kNormThreads * 16) + uint32_t(array * NV + j) * (kNormThreads * 16);
    }
    // `first` points at this thread's vector 0 of the row.  Foreign elements
    // before the row belong to the matrix (a row that does not start on a
    // boundary has one before it); those after it are not read.
    __device__ void fill(int slot, int array, const char *first) const
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (some(j)) {
                const int in = width - col(j);
                cp_async_16(at(slot, array, j), first + j * hop,
                            EXACT || in >= V ? 16u : uint32_t(in) * uint32_t(sizeof(T)));
            }
        }
    }
    // Vector j as pairs of fp32 values, foreign elements as zeros.
    __device__ void read(int slot, int array, int j, F2 (&f)[V / 2]) const
    {
        unpack16<T>(ld_shared_v4(at(slot, array, j)), f);
        clear(j, f);
    }
    __device__ void clear(int j, F2 (&f)[V / 2]) const
    {
        if (!whole(j)) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const float2 v = split(f[e]);
                f[e] = f2(valid(j, 2 * e) ? v.x : 0.f, valid(j, 2 * e + 1) ? v.y : 0.f);
            }
        }
    }
    __device__ void write(char *first, int j, const F2 (&f)[V / 2]) const
    {
        const uint4 q = pack16<T>(f);
        if (whole(j)) {
            *reinterpret_cast<uint4 *>(first + j * hop) = q;
        } else {
            Pack<T, V> o;
            o.q = q;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (valid(j, e)) reinterpret_cast<T *>(first + j * hop)[e] = o.v[e];
        }
    }
    // Weights kept in shared memory behind the rows, each thread its own.
    __device__ uint32_t kept_at(int which, int j, int e) const
    {
        return base + kBytes + uint32_t((which * NV + j) * (V / 4) + e / 2) * (kNormThreads * 16);
    }
    __device__ void keep(int which, int j, const F2 (&f)[V / 2]) const
    {
#pragma unroll
        for (int e = 0; e < V / 2; e += 2) {
            const float2 a = split(f[e]), b = split(f[e + 1]);
            st_shared_v4(kept_at(which, j, e), __float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                         __float_as_uint(b.y));
        }
    }
    __device__ void kept(int which, int j, F2 (&f)[V / 2]) const
    {
#pragma unroll
        for (int e = 0; e < V / 2; e += 2) {
            const float4 q = ld_shared_v4f(kept_at(which, j, e));
            f[e] = f2(q.x, q.y);
            f[e + 1] = f2(q.z, q.w);
        }
    }
    // Weights of vector j, of type T or (f32) fp32; `other` where none are given, 0 for foreign columns.
    __device__ void weights(const void *w, bool f32, float other, int j, F2 (&f)[V / 2]) const
    {
        if (EXACT && w && some(j) && reinterpret_cast<uintptr_t>(w) % 16 == 0) {
            float v[V];
            load_weights<T, V>(w, col(j), f32, v);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) f[e] = f2(v[2 * e], v[2 * e + 1]);
            return;
        }
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            float v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = col(j) + 2 * e + i;
                v[i] = !(some(j) && valid(j, 2 * e + i)) ? 0.f
                       : !w                              ? other
                       : f32                             ? static_cast<const float *>(w)[c]
                                                         : to_f32(static_cast<const T *>(w)[c]);
            }
            f[e] = f2(v[0], v[1]);
        }
    }
};

// Sums over a group's warps of two or four values a thread.  The warps meet on
// a hardware barrier; `buf` holds four values per warp, 8 entries at least for
// each group, those past its warps zero.  Sums that follow one another use two
// buffers: a warp writes a buffer again only after a barrier that every warp of
// the group reaches once it has read it.
struct GroupSums {
    static constexpr int kEntries = kNormThreads / 32 / 2 * 8;  // of groups of 2 warps and more
    uint32_t buf;
    int warps, warp, bar;

    // `mem`: 2 x kEntries entries of the CTA, which this zeroes; every thread calls it.
    __device__ GroupSums(float4 *mem, int warps_) : warps(warps_)
    {
        const int w = int(threadIdx.x) / 32, g = w / warps;
        warp = w - g * warps;
        bar = 1 + g;
        for (int i = int(threadIdx.x); i < 2 * kEntries; i += kNormThreads) mem[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        buf = smem_addr(mem + (warps > 1 ? g * (warps > 8 ? warps : 8) : 0));
        __syncthreads();
    }
    __device__ float4 operator()(float4 v, int which) const
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
            v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
            v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
        }
        if (warps == 1) return v;
        const uint32_t at = buf + uint32_t(which) * (kEntries * 16);
        if ((threadIdx.x & 31u) == 0)
            st_shared_v4(at + uint32_t(warp) * 16, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                         __float_as_uint(v.w));
        named_bar_sync(uint32_t(bar), uint32_t(warps) * 32u);
        F2 a = f2(0.f), b = f2(0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i == 8 && warps <= 8) break;
            const float4 q = ld_shared_v4f(at + uint32_t(i) * 16);
            a = a + f2(q.x, q.y);
            b = b + f2(q.z, q.w);
        }
        const float2 lo = split(a), hi = split(b);
        return make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    __device__ float2 operator()(float x, float y, int which) const
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, o);
            y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        if (warps == 1) return make_float2(x, y);
        // entries of 8 bytes in the same space
        const uint32_t at = buf + uint32_t(which) * (kEntries * 16);
        if ((threadIdx.x & 31u) == 0)
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at + uint32_t(warp) * 8), "f"(x), "f"(y) : "memory");
        named_bar_sync(uint32_t(bar), uint32_t(warps) * 32u);
        F2 a = f2(0.f), b = f2(0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i == 4 && warps <= 8) break;
            const float4 q = ld_shared_v4f(at + uint32_t(i) * 16);
            a = a + f2(q.x, q.y);
            b = b + f2(q.z, q.w);
        }
        return split(a + b);
    }
};

// Shapes of the persistent kernels, by the registers and the shared memory that
// a thread's NV vectors of ARRAYS tensors take.  kPair rows of a group go
// through a step together, where the shared memory holds two steps' rows.  Weights that are
// too many for the registers (32 a thread) are kept in shared memory as fp32: the
// backward pass's, and both of the forward pass's rows of 16 bits; those of fp32
// rows would leave room for one row and are read anew for each (2000 rows of
// 16384 fp16: forward 32.5 to 34 us against 42.3 with weights read anew, backward 52.3
// against 81.2).
template <class T, int NV, int ARRAYS>
struct RowsShape {
    static constexpr bool kWide = NV * 16 / int(sizeof(T)) > 16;
    static constexpr bool kKept = kWide && (ARRAYS == 2 || sizeof(T) == 2);
    static constexpr uint32_t kKeptBytes = kKept ? (ARRAYS == 1 ? 2 : 1) * uint32_t(NV) * 16 / sizeof(T) * kNormThreads * 4 : 0;
    static constexpr int kPerSm = NV == 1 && ARRAYS == 1 ? 2 : 1;                      // CTAs per SM
    static constexpr int kFit = int(192 * 1024 - kKeptBytes) / (NV * ARRAYS * kNormThreads * 16);  // rows of a group
    static constexpr int kPair = kWide || kFit < 4 ? 1 : 2;
    static constexpr int kRows = kFit > 8 ? 8 : kFit / kPair * kPair;
    static_assert(kRows >= kPair, "a step's rows fit");
};

template <class T, int NV, bool EXACT>
__global__ void __launch_bounds__(kNormThreads, RowsShape<T, NV, 1>::kPerSm) norm_fwd_rows_kernel(const NormFwd a, int warps)
{
    constexpr int V = 16 / int(sizeof(T)), ST = RowsShape<T, NV, 1>::kRows;
    constexpr int kPair = RowsShape<T, NV, 1>::kPair;
    constexpr bool kWide = RowsShape<T, NV, 1>::kWide, kKept = RowsShape<T, NV, 1>::kKept;
    __shared__ float4 sums[2 * GroupSums::kEntries];
    extern __shared__ __align__(16) uint8_t mem[];
    const GroupSums total(sums, warps);
    const int groups = kNormThreads / 32 / warps;
    const int64_t row0 = int64_t(blockIdx.x) * groups + int(threadIdx.x) / 32 / warps;
    const int64_t step = int64_t(gridDim.x) * groups;
    const RowRing<T, NV, ST, 1, EXACT> ring(mem, warps, int(a.width), int(uint64_t(row0) * uint64_t(a.ldx) % V));
    const char *x = reinterpret_cast<const char *>(static_cast<const T *>(a.x) + row0 * a.ldx + ring.col(0));
    char *y = reinterpret_cast<char *>(static_cast<T *>(a.y) + row0 * a.ldy + ring.col(0));
    const int64_t x_step = step * a.ldx * int64_t(sizeof(T)), y_step = step * a.ldy * int64_t(sizeof(T));
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll
    for (int k = 0; k < ST; ++k) {
        if (row0 + k * step < a.rows) ring.fill(k, 0, x);
        x += x_step;
        if (k % kPair == kPair - 1) cp_async_commit();
    }
    F2 w[kWide ? 1 : NV][V / 2], b[kWide ? 1 : NV][V / 2];
    if constexpr (!kWide) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            ring.weights(a.w, a.w_f32, 1.f, j, w[j]);
            ring.weights(a.b, a.w_f32, 0.f, j, b[j]);
        }
    } else if constexpr (kKept) {
#pragma unroll 1
        for (int j = 0; j < NV; ++j) {
            ring.weights(a.w, a.w_f32, 1.f, j, w[0]);
            ring.weights(a.b, a.w_f32, 0.f, j, b[0]);
            ring.keep(0, j, w[0]);
            ring.keep(1, j, b[0]);
        }
    }
    int slot = 0;
    for (int64_t row = row0; row < a.rows; row += kPair * step) {
        const bool both = kPair == 2 && row + step < a.rows;
        cp_async_wait<ST / kPair - 1>();
        F2 v[kPair][NV][V / 2];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
            if (h && !both) break;
            F2 s = f2(0.f), s_ = f2(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!ring.some(j)) continue;
                ring.read(slot + h, 0, j, v[h][j]);
#pragma unroll
                for (int e = 0; e < V / 2; e += 2) {
                    s = s + v[h][j][e];
                    s_ = s_ + v[h][j][e + 1];
                }
            }
            sum[h] = sum2(s + s_);
        }
        const float2 total1 = total(sum[0], sum[1], 0);
        const float mean[2] = {total1.x * a.inv_width, total1.y * a.inv_width};
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
            if (row + (ST + h) * step < a.rows) ring.fill(slot + h, 0, x);
            x += x_step;
        }
        cp_async_commit();
        slot = slot + kPair == ST ? 0 : slot + kPair;
        sum[0] = sum[1] = 0.f;
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
            if (h && !both) break;
            const F2 minus = f2(-mean[h]);
            F2 s = f2(0.f), s_ = f2(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!ring.some(j)) continue;
#pragma unroll
                for (int e = 0; e < V / 2; ++e) v[h][j][e] = v[h][j][e] + minus;
                ring.clear(j, v[h][j]);
#pragma unroll
                for (int e = 0; e < V / 2; e += 2) {
                    s = fma2(v[h][j][e], v[h][j][e], s);
                    s_ = fma2(v[h][j][e + 1], v[h][j][e + 1], s_);
                }
            }
            sum[h] = sum2(s + s_);
        }
        const float2 total2 = total(sum[0], sum[1], 1);
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
            if (h && !both) break;
            const float r = 1.f / sqrtf((h ? total2.y : total2.x) * a.inv_width + a.eps);
            if (ring.t == 0) {
                if (a.mean) a.mean[row + h * step] = mean[h];
                if (a.rstd) a.rstd[row + h * step] = r;
            }
            const F2 rr = f2(r);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!ring.some(j)) continue;
                const int k = kWide ? 0 : j;
                if constexpr (kKept) {
                    ring.kept(0, j, w[0]);
                    ring.kept(1, j, b[0]);
                } else if constexpr (kWide) {
                    ring.weights(a.w, a.w_f32, 1.f, j, w[0]);
                    ring.weights(a.b, a.w_f32, 0.f, j, b[0]);
                }
#pragma unroll
                for (int e = 0; e < V / 2; ++e) v[h][j][e] = fma2(v[h][j][e] * rr, w[k][e], b[k][e]);
                ring.write(y, j, v[h][j]);
            }
            y += y_step;
        }
    }
}

// Backward: two sums a row, and each thread's running sums of dy xh and dy over
// its group's rows.  At the end the CTA's groups add theirs in shared memory in
// group order, and the CTA writes one partial row of each.
template <class T, int NV, bool EXACT>
__global__ void __launch_bounds__(kNormThreads, 1) norm_bwd_rows_kernel(const NormBwd a, int warps)
{
    constexpr int V = 16 / int(sizeof(T)), ST = RowsShape<T, NV, 2>::kRows;
    constexpr int kPair = RowsShape<T, NV, 2>::kPair;
    constexpr bool kWide = RowsShape<T, NV, 2>::kWide;  // weights in shared memory
    __shared__ float4 row_sums[2 * GroupSums::kEntries];
    extern __shared__ __align__(16) uint8_t mem[];
    const GroupSums total(row_sums, warps);
    const int groups = kNormThreads / 32 / warps;
    const int g = int(threadIdx.x) / 32 / warps;
    const int64_t row0 = int64_t(blockIdx.x) * groups + g, step = int64_t(gridDim.x) * groups;
    const RowRing<T, NV, ST, 2, EXACT> ring(mem, warps, int(a.width), int(uint64_t(row0) * uint64_t(a.ldx) % V));
    const char *x = reinterpret_cast<const char *>(static_cast<const T *>(a.x) + row0 * a.ldx + ring.col(0));
    const char *dy = reinterpret_cast<const char *>(static_cast<const T *>(a.dy) + row0 * a.lddy + ring.col(0));
    char *dx = reinterpret_cast<char *>(static_cast<T *>(a.dx) + row0 * a.lddx + ring.col(0));
    const int64_t x_step = step * a.ldx * int64_t(sizeof(T)), dy_step = step * a.lddy * int64_t(sizeof(T));
    const int64_t dx_step = step * a.lddx * int64_t(sizeof(T));
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll
    for (int k = 0; k < ST; ++k) {
        if (row0 + k * step < a.rows) {
            ring.fill(k, 0, x);
            ring.fill(k, 1, dy);
        }
        x += x_step;
        dy += dy_step;
        if (k % kPair == kPair - 1) cp_async_commit();
    }
    F2 w[kWide ? 1 : NV][V / 2], dw[NV][V / 2], db[NV][V / 2];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if constexpr (!kWide) ring.weights(a.w, a.w_f32, 1.f, j, w[j]);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) dw[j][e] = db[j][e] = f2(0.f);
    }
    if constexpr (kWide) {
#pragma unroll 1
        for (int j = 0; j < NV; ++j) {
            ring.weights(a.w, a.w_f32, 1.f, j, w[0]);
            ring.keep(0, j, w[0]);
        }
    }
    // The statistics of 32 rows at a time, one row a lane, a batch ahead.
    const int lane = int(threadIdx.x) % 32;
    auto stat = [&](const float *p, int64_t k) {
        const int64_t row = row0 + (k + lane) * step;
        return row < a.rows ? p[row] : 0.f;
    };
    float mean32 = 0.f, rstd32 = 0.f, mean_next = stat(a.mean, 0), rstd_next = stat(a.rstd, 0);
    int slot = 0, flip = 0, k = 0;
    for (int64_t row = row0; row < a.rows; row += kPair * step, k += kPair) {
        if (k % 32 == 0) {
            mean32 = mean_next;
            rstd32 = rstd_next;
            mean_next = stat(a.mean, int64_t(k) + 32);
            rstd_next = stat(a.rstd, int64_t(k) + 32);
        }
        const bool both = kPair == 2 && row + step < a.rows;
        cp_async_wait<ST / kPair - 1>();
        float mean[2], r[2];
        F2 s1[2] = {f2(0.f), f2(0.f)}, s2[2] = {f2(0.f), f2(0.f)};
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
            mean[h] = __shfl_sync(0xffffffffu, mean32, k % 32 + h);
            r[h] = __shfl_sync(0xffffffffu, rstd32, k % 32 + h);
            if (h && !both) break;
            const F2 minus = f2(-mean[h]), rr = f2(r[h]);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!ring.some(j)) continue;
                F2 v[V / 2], d[V / 2];  // d is 0 in foreign columns, so that their v does not count
                ring.read(slot + h, 0, j, v);
                ring.read(slot + h, 1, j, d);
                const int i = kWide ? 0 : j;
                if constexpr (kWide) ring.kept(0, j, w[0]);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const F2 xh = (v[e] + minus) * rr, q = d[e] * w[i][e];
                    dw[j][e] = fma2(d[e], xh, dw[j][e]);
                    db[j][e] = db[j][e] + d[e];
                    s1[h] = s1[h] + q;
                    s2[h] = fma2(q, xh, s2[h]);
                }
            }
        }
        const float4 s = total(make_float4(sum2(s1[0]), sum2(s2[0]), sum2(s1[1]), sum2(s2[1])), flip);
        flip ^= 1;
        // dx = r q - r mean(q) - r mean(q xh) xh, from the rows read once more
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
            if (h && !both) break;
            const F2 minus = f2(-mean[h]), rr = f2(r[h]);
            const F2 c1 = f2(-r[h] * ((h ? s.z : s.x) * a.inv_width)), c2 = f2(-r[h] * ((h ? s.w : s.y) * a.inv_width));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!ring.some(j)) continue;
                F2 v[V / 2], d[V / 2];
                ring.read(slot + h, 0, j, v);
                ring.read(slot + h, 1, j, d);
                const int i = kWide ? 0 : j;
                if constexpr (kWide) ring.kept(0, j, w[0]);
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    d[e] = fma2((v[e] + minus) * rr, c2, fma2(d[e] * w[i][e], rr, c1));
                ring.write(dx, j, d);
            }
            dx += dx_step;
        }
#pragma unroll
        for (int h = 0; h < kPair; ++h) {
            if (row + (ST + h) * step < a.rows) {
                ring.fill(slot + h, 0, x);
                ring.fill(slot + h, 1, dy);
            }
            x += x_step;
            dy += dy_step;
        }
        cp_async_commit();
        slot = slot + kPair == ST ? 0 : slot + kPair;
    }
    if (!a.part) return;
    float *pw = a.part + int64_t(blockIdx.x) * a.width, *pb = pw + int64_t(a.parts) * a.width;
    // Each group's sums in shared memory, in its own vectors' places (column c at
    // c + the group's shift); then every column's groups in group order.
    constexpr uint32_t kHalf = uint32_t(NV) * V * kNormThreads * 4;  // bytes of all groups' sums of one kind
    const uint32_t each = uint32_t(ring.threads) * NV * V * 4;       // and of one group's
    cp_async_wait<0>();
    __syncthreads();  // every thread is done with its rows' shared memory
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t at = smem_addr(mem) + uint32_t(g) * each + uint32_t((ring.t + j * ring.threads) * V) * 4u;
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float2 w0 = split(dw[j][e / 2]), w1 = split(dw[j][e / 2 + 1]);
            const float2 b0 = split(db[j][e / 2]), b1 = split(db[j][e / 2 + 1]);
            st_shared_v4(at + uint32_t(e) * 4u, __float_as_uint(w0.x), __float_as_uint(w0.y), __float_as_uint(w1.x),
                         __float_as_uint(w1.y));
            st_shared_v4(at + kHalf + uint32_t(e) * 4u, __float_as_uint(b0.x), __float_as_uint(b0.y),
                         __float_as_uint(b1.x), __float_as_uint(b1.y));
        }
    }
    __syncthreads();
    for (int c = int(threadIdx.x); c < int(a.width); c += kNormThreads) {
        float vw = 0.f, vb = 0.f;
        for (int i = 0; i < groups; ++i) {
            const int64_t first = int64_t(blockIdx.x) * groups + i;  // the group's first row
            if (first >= a.rows) break;
            const int shift = EXACT ? 0 : int(uint64_t(first) * uint64_t(a.ldx) % V);
            const float *at = reinterpret_cast<const float *>(mem + uint32_t(i) * each) + c + shift;
            vw += at[0];
            vb += at[kHalf / 4];
        }
        pw[c] = vw;
        pb[c] = vb;
    }
}

// ---------------------------------------------------------------- wide rows

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

// Adds the partial rows of dw (blockIdx.y 0) and db (1): 32 columns a CTA, whose
// warps (up to 32) take parts w, w + warps, ...; the warps' sums are added in a
// fixed tree.
template <class W>
__global__ void __launch_bounds__(1024) norm_bwd_reduce_kernel(const float *part, int parts, int64_t width, W *dw, W *db)
{
    __shared__ float s[32][33];
    W *out = blockIdx.y ? db : dw;
    const float *p = part + int64_t(blockIdx.y) * parts * width;
    const int lane = int(threadIdx.x) % 32, w = int(threadIdx.x) / 32, warps = int(blockDim.x) / 32;
    const int64_t c0 = int64_t(blockIdx.x) * 32, c = c0 + lane;
    griddep_wait();
    griddep_launch_dependents();
    if (!out) return;
    float v = 0.f;
    if (c < width) {
#pragma unroll 8
        for (int i = w; i < parts; i += warps) v += p[int64_t(i) * width + c];
    }
    if (warps == 1) {
        if (c < width) out[c] = from_f32<W>(v);
        return;
    }
    s[w][lane] = v;
    __syncthreads();
    for (int i = w; i < 32; i += warps) {  // column i's sums of the warps, a lane each
        const float total = warp_sum(lane < warps ? s[lane][i] : 0.f);
        if (lane == 0 && c0 + i < width) out[c0 + i] = from_f32<W>(total);
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

template <class T, int NV>
static int fwd_launch(const NormFwd &a, int warps, cudaStream_t s)
{
    if (warps > 1) return launch(norm_fwd_kernel<T, NV, true>, dim3(unsigned(a.rows)), dim3(unsigned(32 * warps)), 0, s, 1, a);
    return launch(norm_fwd_kernel<T, NV, false>, dim3(unsigned((a.rows + 3) / 4)), dim3(128), 0, s, 1, a);
}

template <class T, int NV>
static int fwd_vec_launch(const NormFwd &a, int warps, cudaStream_t s)
{
    const dim3 grid(unsigned(a.rows)), block(unsigned(32 * warps));
    if (warps > 16) return launch(norm_fwd_vec_kernel<T, NV, true, 1024>, grid, block, 0, s, 1, a);
    if (warps > 8) return launch(norm_fwd_vec_kernel<T, NV, true, 512>, grid, block, 0, s, 1, a);
    if (warps > 1) return launch(norm_fwd_vec_kernel<T, NV, true, 256>, grid, block, 0, s, 1, a);
    return launch(norm_fwd_vec_kernel<T, NV, false, 256>, dim3(unsigned((a.rows + 7) / 8)), dim3(256), 0, s, 1, a);
}

// Dynamic shared memory above 48 KB has to be allowed per kernel and device.
static int allow_smem(const void *kernel, size_t bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    if (bytes <= 48 * 1024) return kOk;
    if (cudaGetDevice(&dev) != cudaSuccess) return kErrCuda;
    if (dev < 64 && (done.load() >> dev & 1)) return kOk;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) != cudaSuccess) {
        cudaGetLastError();
        return kErrCuda;
    }
    if (dev < 64) done.fetch_or(uint64_t(1) << dev);
    return kOk;
}

// CTAs of a persistent launch per CTA slot of an SM: a multiple of 8, so that a
// group's rows share one shift.
static int row_ctas(int sms) { return sms / 8 * 8; }

// Groups and vectors per thread for the persistent kernels: up to 16 elements
// a thread, in as few warps as that allows; 32 in rows wider than 16 warps hold
// that way.
template <class T>
static bool rows_shape(int64_t width, int64_t ld, int *warps, int *nv)
{
    constexpr int V = 16 / int(sizeof(T));
    const int64_t worst_shift = ld % V ? V - 1 : 0;
    return row_shape((width + worst_shift + V - 1) / V, 16 / V, 32 / V, kNormThreads / 32, warps, nv);
}

template <class T, int NV, bool EXACT>
static int fwd_rows_launch(const NormFwd &a, int warps, int sms, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem =
        RowRing<T, NV, RowsShape<T, NV, 1>::kRows, 1, EXACT>::kBytes + RowsShape<T, NV, 1>::kKeptBytes;
    const int rc = allow_smem(reinterpret_cast<const void *>(&norm_fwd_rows_kernel<T, NV, EXACT>), smem, done);
    if (rc != kOk) return rc;
    return launch(norm_fwd_rows_kernel<T, NV, EXACT>, dim3(unsigned(row_ctas(sms) * RowsShape<T, NV, 1>::kPerSm)),
                  dim3(kNormThreads), smem, s, 1, a, warps);
}

// vec: rows of whole 16-byte vectors throughout; shifted: the first rows of x
// and y start on a 16-byte boundary and later ones equally far from one.
template <class T>
static int fwd(const NormFwd &a, bool vec, bool shifted, int sms, cudaStream_t s)
{
    constexpr int V = 16 / int(sizeof(T));
    const bool exact = a.width % V == 0 && a.ldx % V == 0;
    int warps = 0, nv = 0;
    // Many rows: the persistent form.  Few: a CTA (or warp) of its own for each row.
    if (shifted && row_ctas(sms) > 0 && rows_shape<T>(a.width, a.ldx, &warps, &nv) &&
        a.rows >= int64_t(warps < 16 ? 8 : nv * V > 16 ? 1 : 4) * sms * (kNormThreads / 32 / warps)) {
        if (nv == 1) return exact ? fwd_rows_launch<T, 1, true>(a, warps, sms, s)
                            : fwd_rows_launch<T, 1, false>(a, warps, sms, s);
        if (nv == 2) return exact ? fwd_rows_launch<T, 2, true>(a, warps, sms, s)
                            : fwd_rows_launch<T, 2, false>(a, warps, sms, s);
        if (nv == 4)
            return exact ? fwd_rows_launch<T, 4, true>(a, warps, sms, s) : fwd_rows_launch<T, 4, false>(a, warps, sms, s);
        if constexpr (V == 4)
            return exact ? fwd_rows_launch<T, 8, true>(a, warps, sms, s) : fwd_rows_launch<T, 8, false>(a, warps, sms, s);
    }
    if (vec && row_shape(a.width / V, 16 / V, 16 / V, 32, &warps, &nv)) {
        if (nv == 1) return fwd_vec_launch<T, 1>(a, warps, s);
        if (nv == 2) return fwd_vec_launch<T, 2>(a, warps, s);
        if constexpr (V == 4) return fwd_vec_launch<T, 4>(a, warps, s);
    }
    if (row_shape(a.width, 16, 16, 32, &warps, &nv)) {
        switch (nv) {
        case 1: return fwd_launch<T, 1>(a, warps, s);
        case 2: return fwd_launch<T, 2>(a, warps, s);
        case 4: return fwd_launch<T, 4>(a, warps, s);
        case 8: return fwd_launch<T, 8>(a, warps, s);
        default: return fwd_launch<T, 16>(a, warps, s);
        }
    }
    return launch(norm_fwd_wide_kernel<T>, dim3(unsigned(a.rows)), dim3(1024), 0, s, 1, a);
}

// CTAs (and partial rows) of the backward pass.
static int bwd_parts(int64_t rows, int sms)
{
    const int most = row_ctas(sms) ? row_ctas(sms) : sms;
    return rows < 1 ? 1 : rows < most ? int(rows) : most;
}

template <class T, int NV, bool EXACT>
static int bwd_rows_launch(const NormBwd &a, int warps, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    constexpr size_t ring = RowRing<T, NV, RowsShape<T, NV, 2>::kRows, 2, EXACT>::kBytes;
    static_assert(ring >= 2 * size_t(NV) * 16 / sizeof(T) * kNormThreads * 4,
                  "the groups' sums fit the rows' shared memory");
    constexpr size_t smem = ring + RowsShape<T, NV, 2>::kKeptBytes;
    const int rc = allow_smem(reinterpret_cast<const void *>(&norm_bwd_rows_kernel<T, NV, EXACT>), smem, done);
    if (rc != kOk) return rc;
    return launch(norm_bwd_rows_kernel<T, NV, EXACT>, dim3(unsigned(a.parts)), dim3(kNormThreads), smem, s, 1, a, warps);
}

template <class T>
static int bwd(const NormBwd &a, bool shifted, int sms, cudaStream_t s)
{
    constexpr int V = 16 / int(sizeof(T));
    const bool exact = a.width % V == 0 && a.ldx % V == 0;
    int warps = 0, nv = 0;
    // One row a group, or (a.parts a multiple of 8) rows that share a shift.
    if (shifted && (a.rows <= a.parts || row_ctas(sms) > 0) && rows_shape<T>(a.width, a.ldx, &warps, &nv)) {
        if (nv == 1) return exact ? bwd_rows_launch<T, 1, true>(a, warps, s)
                            : bwd_rows_launch<T, 1, false>(a, warps, s);
        if (nv == 2) return exact ? bwd_rows_launch<T, 2, true>(a, warps, s)
                            : bwd_rows_launch<T, 2, false>(a, warps, s);
        if (nv == 4)
            return exact ? bwd_rows_launch<T, 4, true>(a, warps, s) : bwd_rows_launch<T, 4, false>(a, warps, s);
        if constexpr (V == 4)
            return exact ? bwd_rows_launch<T, 8, true>(a, warps, s) : bwd_rows_launch<T, 8, false>(a, warps, s);
    }
    // The column sums first: dx may take the place of dy or x.
    if (a.part) {
        const int rc = launch(norm_bwd_cols_kernel<T>, dim3(unsigned((a.width + 255) / 256), unsigned(a.parts)), dim3(256),
                              0, s, 1, a);
        if (rc != kOk) return rc;
    }
    return launch(norm_bwd_wide_kernel<T>, dim3(unsigned(a.rows)), dim3(1024), 0, s, 1, a);
}

template <class W>
static int reduce(const NormBwd &a, void *dw, void *db, cudaStream_t s)
{
    const unsigned warps = a.parts < 32 ? unsigned(a.parts) : 32u;
    return launch(norm_bwd_reduce_kernel<W>, dim3(unsigned((a.width + 31) / 32), 2), dim3(32 * warps), 0, s, 1,
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
    const bool shifted = aligned16(x) && aligned16(y) && (ldx - ldy) * e % 16 == 0;
    const bool vec = shifted && aligned16(weight) && aligned16(bias) && ldx * e % 16 == 0 && width * e % 16 == 0;
    const NormFwd a{rows, width, ldx, ldy, x, weight, bias, y, mean, rstd, eps, float(1.0 / double(width)),
                    weight_dtype == kF32};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == kF32) return fwd<float>(a, vec, shifted, d.sms, s);
    return dtype == kF16 ? fwd<__half>(a, vec, shifted, d.sms, s)
                         : fwd<__nv_bfloat16>(a, vec, shifted, d.sms, s);
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
    const bool shifted = aligned16(dy) && aligned16(x) && aligned16(dx) && (ldx - lddy) * e % 16 == 0 &&
                         (ldx - lddx) * e % 16 == 0;
    const NormBwd a{rows, width, lddy, ldx, lddx, dy, x, weight, mean, rstd, dx,
                    sums ? static_cast<float *>(workspace) : nullptr, parts, float(1.0 / double(width)),
                    weight_dtype == kF32};
    rc = dtype == kF32   ? bwd<float>(a, shifted, d.sms, s)
         : dtype == kF16 ? bwd<__half>(a, shifted, d.sms, s)
                         : bwd<__nv_bfloat16>(a, shifted, d.sms, s);
    if (rc != kOk || !sums) return rc;
    if (weight_dtype == kF32) return reduce<float>(a, dweight, dbias, s);
    return weight_dtype == kF16 ? reduce<__half>(a, dweight, dbias, s) : reduce<__nv_bfloat16>(a, dweight, dbias, s);
}

}  // extern "C"
