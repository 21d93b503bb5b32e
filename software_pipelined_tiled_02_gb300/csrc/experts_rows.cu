// experts_rows.cu -- the work around the experts' products: the order of pairs by
// expert, rows gathered into it, and each token's sum over its pairs.
//
// Nothing here depends on timing: a pair's place follows from the counts of
// experts before it, and every sum runs in the pairs' order.
//
// What bounds it: bytes.  8192 tokens, 4 of 32 experts, 4096 wide: gathering reads 67
// MB (and the same rows again from L2) and writes 268 in 65 us, combining reads 537 MB
// of fp32 and writes 67 in 92 us, 6.6 TB/s.  Placing takes 8 us and counting 5, of which
// launches overlap most.  Loading the rows in the product itself, four at a time by
// their indices, would save the gathered copy, but the copy engine takes 30 ns for four
// rows: Up took 2.4 ms instead of 0.7.

#include <cuda_runtime.h>

#include "elem.cuh"
#include "experts.cuh"
#include "host.h"
#include "ptx.cuh"

namespace tg {

constexpr int kPlaceThreads = 256, kPlaceWarps = kPlaceThreads / 32;
constexpr int kPairsPerWarp = kChunkPairs / kPlaceWarps;

// Pairs of each expert in one chunk.
__global__ void __launch_bounds__(kPlaceThreads) experts_count_kernel(const int *chosen, int64_t pairs, int experts, int *counts)
{
    __shared__ int seen[kMostExperts];
    for (int e = int(threadIdx.x); e < experts; e += kPlaceThreads) seen[e] = 0;
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * kChunkPairs;
    for (int i = int(threadIdx.x); i < kChunkPairs && first + i < pairs; i += kPlaceThreads) {
        const int e = chosen[first + i];
        if (e >= 0 && e < experts) atomicAdd(&seen[e], 1);
    }
    __syncthreads();
    for (int e = int(threadIdx.x); e < experts; e += kPlaceThreads) counts[int64_t(blockIdx.x) * experts + e] = seen[e];
}

// Exclusive sums of a, b and c over the CTA's threads; the totals in `all`.
__device__ __forceinline__ void scan3(int &a, int &b, int &c, int (&all)[3])
{
    __shared__ int warps[kPlaceWarps][3];
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32;
    int v[3] = {a, b, c}, mine[3] = {a, b, c};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int up = __shfl_up_sync(0xffffffffu, v[k], o);
            if (lane >= o) v[k] += up;
        }
    __syncthreads();
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < 3; ++k) warps[warp][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        int before = 0, total = 0;
        for (int w = 0; w < kPlaceWarps; ++w) {
            if (w < warp) before += warps[w][k];
            total += warps[w][k];
        }
        v[k] += before - mine[k];
        all[k] = total;
    }
    a = v[0];
    b = v[1];
    c = v[2];
}

// Many counts: an expert's become the pairs before each chunk, and the row behind the
// last chunk takes them all.  One CTA an expert.  Without it every placing CTA reads all
// counts: a forward pass of 64 x 64 experts, pairs x experts 32768 x 32: 37.4 us so, 37.9
// with this kernel; 65536 x 256: 73 and 61; 1048576 x 256: 1070 and 593.
__global__ void __launch_bounds__(kPlaceThreads) experts_scan_kernel(int *counts, int chunks, int experts)
{
    griddep_wait();
    griddep_launch_dependents();
    int *of = counts + blockIdx.x;
    int before = 0;
    for (int c0 = 0; c0 < chunks; c0 += kPlaceThreads) {
        const int c = c0 + int(threadIdx.x);
        int n = c < chunks ? of[int64_t(c) * experts] : 0, unused[2] = {0, 0}, all[3];
        scan3(n, unused[0], unused[1], all);
        if (c < chunks) of[int64_t(c) * experts] = before + n;
        before += all[0];
    }
    if (threadIdx.x == 0) of[int64_t(chunks) * experts] = before;
}

// One chunk's pairs to their rows.  A warp takes kPairsPerWarp neighbours, 32 at a
// time; lanes with the same expert find each other.  The first CTA also writes
// the offsets, the row tiles and the filling.
__global__ void __launch_bounds__(kPlaceThreads)
    experts_place_kernel(const int *chosen, int64_t pairs, int experts, int chunks, bool scanned, const Placed p)
{
    extern __shared__ int smem[];
    int *next = smem;                               // [warps][experts] rows handed out next
    int *total = smem + kPlaceWarps * experts;      // [experts] pairs of all chunks
    int *earlier = smem + (kPlaceWarps + 1) * experts;  // [experts] pairs of the chunks before this one
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32;
    for (int i = int(threadIdx.x); i < (kPlaceWarps + 2) * experts; i += kPlaceThreads) next[i] = 0;
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * kChunkPairs + warp * kPairsPerWarp;
    int mine[kPairsPerWarp / 32];
#pragma unroll
    for (int r = 0; r < kPairsPerWarp / 32; ++r) {
        const int64_t i = first + r * 32 + lane;
        int e = i < pairs ? chosen[i] : -1;
        if (e < 0 || e >= experts) e = -1;
        mine[r] = e;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(int(same)) - 1) next[warp * experts + e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // All chunks' counts: scanned, as the counting kernel left them, or for few pairs
    // from the pairs themselves.
    if (scanned) {
        for (int e = int(threadIdx.x); e < experts; e += kPlaceThreads) {
            total[e] = p.counts[int64_t(chunks) * experts + e];
            earlier[e] = p.counts[int64_t(blockIdx.x) * experts + e];
        }
    } else if (p.counts) {
        for (int64_t i = threadIdx.x; i < int64_t(chunks) * experts; i += kPlaceThreads) {
            const int n = p.counts[i], c = int(i / experts), e = int(i - int64_t(c) * experts);
            if (n) atomicAdd(&total[e], n);
            if (n && c < int(blockIdx.x)) atomicAdd(&earlier[e], n);
        }
    } else {
        for (int i = int(threadIdx.x); i < int(pairs); i += kPlaceThreads) {
            const int e = chosen[i];
            if (e < 0 || e >= experts) continue;
            atomicAdd(&total[e], 1);
            if (i / kChunkPairs < int(blockIdx.x)) atomicAdd(&earlier[e], 1);
        }
    }
    __syncthreads();
    // Each thread takes neighbouring experts, so that sums over threads run in the experts' order.
    const int per = (experts + kPlaceThreads - 1) / kPlaceThreads, e0 = int(threadIdx.x) * per;
    int plain = 0, padded = 0, tiles = 0;
    for (int e = e0; e < e0 + per && e < experts; ++e) {
        const int all = total[e];
        plain += all;
        padded += (all + kPadRows - 1) / kPadRows * kPadRows;
        tiles += (all + kRowTile - 1) / kRowTile;
        int before = earlier[e];  // rows before each warp's within the expert
        for (int w = 0; w < kPlaceWarps; ++w) {
            const int n = next[w * experts + e];
            next[w * experts + e] = before;
            before += n;
        }
    }
    int sums[3];
    scan3(plain, padded, tiles, sums);
    for (int e = e0; e < e0 + per && e < experts; ++e) {
        const int n = total[e], filled = (n + kPadRows - 1) / kPadRows * kPadRows;
        for (int w = 0; w < kPlaceWarps; ++w) next[w * experts + e] += padded;
        if (blockIdx.x == 0) {
            p.offsets[e] = plain;
            p.padded[e] = padded;
            for (int r = n; r < filled; ++r) p.pair_of[padded + r] = -1;
            for (int r = 0; r < n; r += kRowTile)
                p.table[tiles + r / kRowTile] = RowTile{e, plain + r, padded + r, min(kRowTile, n - r)};
        }
        plain += n;
        padded += filled;
        tiles += (n + kRowTile - 1) / kRowTile;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.offsets[experts] = sums[0];
        p.padded[experts] = sums[1];
        *p.tiles = sums[2];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPairsPerWarp / 32; ++r) {
        const int64_t i = first + r * 32 + lane;
        const int e = mine[r];
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = next[warp * experts + e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(int(same)) - 1) next[warp * experts + e] += __popc(same);
        __syncwarp();
        if (i < pairs) {
            p.row_of[i] = row;
            if (row >= 0) p.pair_of[row] = int(i);
        }
    }
}

int experts_place(const ExpertSizes &z, const int *chosen, const Placed &p, cudaStream_t s)
{
    const int64_t chunks = chunks_of(z);
    Placed at = p;
    if (z.pairs <= kCountedInPlace) at.counts = nullptr;
    if (at.counts) {
        const int rc = launch(experts_count_kernel, dim3(unsigned(chunks)), dim3(kPlaceThreads), 0, s, 1, chosen, z.pairs,
                              int(z.experts), p.counts);
        if (rc != kOk) return rc;
    }
    const bool scanned = at.counts && chunks * z.experts > kScannedCounts;
    if (scanned) {
        const int rc = launch(experts_scan_kernel, dim3(unsigned(z.experts)), dim3(kPlaceThreads), 0, s, 1, p.counts, int(chunks),
                              int(z.experts));
        if (rc != kOk) return rc;
    }
    return launch(experts_place_kernel, dim3(unsigned(chunks)), dim3(kPlaceThreads), size_t(4 * (kPlaceWarps + 2) * z.experts), s,
                  1, chosen, z.pairs, int(z.experts), int(chunks), scanned, at);
}

// A warp copies one row, 16 bytes a lane and step.
constexpr int kGatherWarps = 8;
__global__ void __launch_bounds__(32 * kGatherWarps) experts_gather_kernel(const Gather g, int vecs, int top, int experts, const Placed p)
{
    const int lane = int(threadIdx.x) % 32;
    griddep_wait();
    griddep_launch_dependents();
    const int rows = p.padded[experts];
    for (int64_t row = int64_t(blockIdx.x) * kGatherWarps + threadIdx.x / 32; row < rows; row += int64_t(gridDim.x) * kGatherWarps) {
        const int pair = p.pair_of[row];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (!g.to[m]) break;
            const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(g.from[m]) + int64_t(pair / top) * g.ld[m]);
            uint4 *to = static_cast<uint4 *>(g.to[m]) + row * vecs;
            int v = lane;
            for (; v + 96 < vecs; v += 128) {
                uint4 q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = pair < 0 ? make_uint4(0u, 0u, 0u, 0u) : from[v + 32 * i];
#pragma unroll
                for (int i = 0; i < 4; ++i) to[v + 32 * i] = q[i];
            }
            for (; v < vecs; v += 32) to[v] = pair < 0 ? make_uint4(0u, 0u, 0u, 0u) : from[v];
        }
    }
}

int experts_gather(const ExpertSizes &z, int64_t width, const Gather &g, const Placed &p, cudaStream_t s)
{
    const int64_t blocks = (z.padded_rows + kGatherWarps - 1) / kGatherWarps;
    return launch(experts_gather_kernel, dim3(unsigned(blocks < 65536 ? blocks : 65536)), dim3(32 * kGatherWarps), 0, s, 1, g,
                  int(width / 8), z.top, int(z.experts), p);
}

// A CTA takes a token's 2048 columns, 8 a thread; each thread adds its columns of
// the token's rows in order.
template <class T>
__global__ void __launch_bounds__(256) experts_combine_kernel(const Combine c, int64_t width, int top, const Placed p)
{
    __shared__ int rows[kMostTop];
    __shared__ float weights[kMostTop];
    const int64_t t = blockIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    if (int(threadIdx.x) < top) {
        const int64_t pair = t * top + threadIdx.x;
        if (c.chosen) {
            const int e = c.chosen[pair];
            rows[threadIdx.x] = e < 0 || e >= c.experts ? -1 : int(pair);
        } else {
            rows[threadIdx.x] = p.row_of[pair];
        }
        weights[threadIdx.x] = c.weights ? c.weights[t * top + threadIdx.x] : 1.f;
    }
    __syncthreads();
    if (c.dweights && blockIdx.y == 0) {
        for (int j = int(threadIdx.x) / 32; j < top; j += 8) {  // a warp a pair
            const int row = rows[j];
            float sum = 0.f;
            if (row >= 0)
                for (int i = int(threadIdx.x) % 32; i < c.nparts; i += 32) sum += c.parts[i * c.part_stride + row];
            sum = warp_sum(sum);
            if (threadIdx.x % 32 == 0) c.dweights[t * top + j] = sum;
        }
    }
    const int64_t col = (int64_t(blockIdx.y) * 256 + threadIdx.x) * 8;
    if (!c.out || col >= width) return;
    F2 sum[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
    for (int j = 0; j < top; ++j) {
        if (rows[j] < 0) continue;
        const uint4 *from = reinterpret_cast<const uint4 *>(c.rows + int64_t(rows[j]) * width + col);
        F2 a[2], b[2];
        unpack16<float>(from[0], a);
        unpack16<float>(from[1], b);
        const F2 w = f2(weights[j]);
        sum[0] = fma2(a[0], w, sum[0]);
        sum[1] = fma2(a[1], w, sum[1]);
        sum[2] = fma2(b[0], w, sum[2]);
        sum[3] = fma2(b[1], w, sum[3]);
    }
    *reinterpret_cast<uint4 *>(static_cast<T *>(c.out) + t * c.ld + col) = pack16<T>(sum);
}

int experts_combine(const ExpertSizes &z, int64_t width, bool bf16, const Combine &c, const Placed &p, cudaStream_t s)
{
    const dim3 grid(unsigned(z.tokens), c.out ? unsigned((width + 2047) / 2048) : 1u);
    return bf16 ? launch(experts_combine_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, 1, c, width, z.top, p)
                : launch(experts_combine_kernel<__half>, grid, dim3(256), 0, s, 1, c, width, z.top, p);
}

}  // namespace tg
