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
//   A nibble becomes a number by its bits alone, as Kim, Henry, Fahim and Awadalla
// (Who Says Elephants Can't Run, 2022) convert integer weights: or-ed into the mantissa of 1024
// (fp16) or 128 (bf16), from which 1024 + z or 128 + z is subtracted, two at a
// time.  A word's nibbles come out as the pairs (0, 4), (1, 5), (2, 6), (3, 7);
// the order of k does not matter to a sum as long as x is taken in the same one,
// so x's pairs are permuted, not the weights.
//
// What bounds it: the SMs, not the memory; weights that lie in L2 take as long (8192 x
// 8192, 12.4 us against 13.5).  One token, 16384 x 8192 in groups of 128 (69 MB, 10.4 us
// at the memory's rate): 21.6 us in bf16, 20.6 in fp16, 3.2 and 3.4 TB/s; 8 tokens 23.1
// and 21.7.  5.4 us are a launch's start and end, and a CTA's 32 rows take 4.2 us of an
// SM: 300 instructions a chunk of 32 x 128 weights, 60 % of the issue slots where four
// CTAs share the SM, and 512 CTAs leave some SMs three.  What was slower: the weights
// straight into registers (30 us), all of k by one warp, with 14 or 28 warps of other
// blocks beside it (28 to 33), 256 bytes of a row at a time (33), four accumulators a
// chunk (23.7), scales read where they lie (26), one CTA of 16 warps an SM that shares
// out its rows evenly but has one chain of steps a warp (25.5), five CTAs an SM in 96
// registers (24).  The warps share out k, copy their own chunks, and add their sums in
// warp order.

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "elem.cuh"
#include "host.h"
#include "pairs.cuh"
#include "ptx.cuh"
#include "tgemm.h"

namespace tg {

struct W4 {
    const uint16_t *x;
    int64_t ldx;
    const uint8_t *packed;
    const void *scales;
    const uint8_t *zeros;   // NULL: 8
    Pairs pairs;            // its experts NULL: one matrix
    void *y;
    int64_t n, k, groups;   // groups of a row
    int64_t group;
    int each;               // rows of y for one row of x
    bool scales_f32, y_f32;
};

// Constants kept in registers, twice 16 bits each.  The compiler would take the
// masking apart into two instructions of an immediate each, and make a sum, for
// which it has the masking's pipe alone, of the product with 1.
struct Nibbles {
    uint32_t mask, base, unit;  // 0x000f, 1024 or 128, 1
    uint32_t mask_up, unit_up;  // fp16: 0x00f0, 1 / 16
};
template <bool BF16>
__device__ __forceinline__ Nibbles nibbles()
{
    Nibbles n;
    asm volatile("mov.b32 %0, %1;" : "=r"(n.mask) : "n"(0x000f000f));
    asm volatile("mov.b32 %0, %1;" : "=r"(n.base) : "n"(BF16 ? 0x43004300 : 0x64006400));
    asm volatile("mov.b32 %0, %1;" : "=r"(n.unit) : "n"(BF16 ? 0x3F803F80 : 0x3C003C00));
    asm volatile("mov.b32 %0, %1;" : "=r"(n.mask_up) : "n"(0x00f000f0));
    asm volatile("mov.b32 %0, %1;" : "=r"(n.unit_up) : "n"(0x2C002C00));
    return n;
}

// 8 nibbles as four pairs of q - z.  `less` holds -(128 + z), or -(1024 + z), twice.  fp16's
// mantissa has room for a nibble at bit 4 too, which makes 1024 + 16 q; a sixteenth
// of it less 64 + z (`less_up`) saves every second shift.
template <bool BF16>
__device__ __forceinline__ void spread(uint32_t w, uint32_t less, uint32_t less_up, const Nibbles &n, uint32_t (&a)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v;
        if constexpr (BF16) {
            asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)), "r"(n.mask), "r"(n.base));  // (w & mask) | base
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(a[i]) : "r"(v), "r"(n.unit), "r"(less));
        } else {
            asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (8 * (i / 2))), "r"(i % 2 ? n.mask_up : n.mask), "r"(n.base));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(a[i]) : "r"(v), "r"(i % 2 ? n.unit_up : n.unit), "r"(i % 2 ? less_up : less));
        }
    }
}

// 8 values of x as a word's nibbles come out: the pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint4 w4_permuted(uint4 q)
{
    return make_uint4(__byte_perm(q.x, q.z, 0x5410), __byte_perm(q.x, q.z, 0x7632), __byte_perm(q.y, q.w, 0x5410),
                      __byte_perm(q.y, q.w, 0x7632));
}

// The shared memory of a CTA: each warp's ring of chunks (later the warps' sums),
// the block's scales in fp32 and its zero points, and (HELD) the tokens' rows of x.
constexpr int kW4Early = 4;               // loads of a kind that a thread has on their way
constexpr int64_t kW4Held = 20 * 1024;    // x is held in shared memory up to this size
constexpr int64_t kW4Scales = 48 * 1024;  // scales and zero points are, up to this size; beyond it they are read where they lie

struct W4Space {
    int pitch;  // of scales and zero points, odd: 8 rows lie in 8 banks; 0: not in shared memory
    int off_zeros, off_x, total;
};
constexpr int kDepth = 2;  // chunks of a warp on their way
template <int WARPS, int NT, int R>
struct W4Ring {
    static constexpr int kRing = WARPS * kDepth * R * 16 * 64, kSums = WARPS * R * 16 * (8 * NT + 1) * 4;
    static constexpr int kBytes = kRing > kSums ? kRing : kSums;
};

// Where 16-byte vector j of a row of x lies: neighbours of 4 are exchanged, so that
// vectors 4 apart do not meet in a bank.
__device__ __forceinline__ unsigned w4_twist(unsigned j) { return j ^ ((j >> 2) & 3u); }

template <bool BF16>
__device__ __forceinline__ float w4_scale(const W4 &p, int64_t i)
{
    if (p.scales_f32) return static_cast<const float *>(p.scales)[i];
    if constexpr (BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.scales)[i]);
    else
        return __half2float(static_cast<const __half *>(p.scales)[i]);
}

// 16 R weight rows and up to 8 NT tokens.  A chunk is 128 weights of each row, of SUB
// groups at least.  A warp's chunks are neighbours, and its copies of them are its
// own, so it waits for nobody until the block is summed.  Columns of tokens that are
// not there repeat the last one's and are dropped.
template <bool BF16, int SUB, int WARPS, int NT, int R, bool HELD>
__global__ void __launch_bounds__(32 * WARPS, NT > 2 ? 1 : 16 / WARPS) w4_kernel(const W4 p, const W4Space sp)
{
    constexpr int kWords = 4 / SUB;                // words of 8 weights that a lane takes of a row and group
    constexpr int kThreads = 32 * WARPS, kPerRow = kThreads / (16 * R);
    constexpr uint32_t kChunkBytes = R * 16 * 64;
    constexpr uint32_t minus = BF16 ? 0xC300C300u : 0xE400E400u;  // -128 or -1024, twice
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int list[8 * NT], listed[2];
    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32, g = lane / 4, c = lane % 4;
    const int64_t row0 = int64_t(blockIdx.x) * (16 * R);
    const Nibbles nib = nibbles<BF16>();
    griddep_wait();

    int expert = 0, from = int(blockIdx.z) * 8 * NT;
    if (p.pairs.experts) {
        if (!slot_expert(p.pairs, int(blockIdx.y), expert)) return;
        from = 0;
    }
    const int k = int(p.k), all_chunks = (k + 127) / 128, each_warp = (all_chunks + WARPS - 1) / WARPS;
    const int chunk0 = min(warp * each_warp, all_chunks);
    const int n_chunks = expert < 0 ? 0 : min(each_warp, all_chunks - chunk0);
    const int64_t matrix_row = int64_t(max(expert, 0)) * p.n + row0;
    const int here = int(min(int64_t(16 * R), p.n - row0));  // rows of the block

    // A lane copies the 16 bytes c of the chunk's rows g, g + 8, ..  They lie in
    // shared memory with c exchanged by g's bits, so that lanes that read other
    // words of the rows (SUB > 1) do not meet in a bank.
    const uint32_t ring = smem_addr(smem) + uint32_t(warp * kDepth) * kChunkBytes;
    const int twist = (g >> 1) & 3;
    const uint32_t ring_to = ring + uint32_t(g * 64 + ((c ^ twist) << 4));
    const uint8_t *weights = p.packed + matrix_row * (p.k / 2) + chunk0 * 64 + c * 16;
    uint32_t rows[2 * R];  // in units of 16 bytes
#pragma unroll
    for (int r = 0; r < 2 * R; ++r) rows[r] = uint32_t(min(r * 8 + g, here - 1)) * uint32_t(k / 32);  // past the last row: computed and dropped
    auto fetch = [&](int slot, int i) {  // the warp's chunk i
        if (i < n_chunks && (SUB == 1 || (chunk0 + i) * 128 + c * 32 < k)) {
#pragma unroll
            for (int r = 0; r < 2 * R; ++r)
                cp_async_16(ring_to + uint32_t(slot) * kChunkBytes + uint32_t(r * 512), weights + uint64_t(rows[r]) * 16 + i * 64, 16);
        }
        cp_async_commit();
    };

    // Scales and zero points: unit q (128 / SUB weights of a row) is in group q / per.
    const int per = int(p.group) / (128 / SUB), groups = int(p.groups), all_groups = sp.pitch && expert >= 0 ? groups : 0;
    float *scales = reinterpret_cast<float *>(smem + W4Ring<WARPS, NT, R>::kBytes);
    uint8_t *zeros = smem + sp.off_zeros;
    const int64_t group_row0 = matrix_row * p.groups;
    auto groups_of = [&](int q, float (&scale)[2 * R], uint32_t (&less)[2 * R], uint32_t (&less_up)[2 * R]) {
        const int at = per == 1 ? q : q / per;
#pragma unroll
        for (int r = 0; r < 2 * R; ++r) {
            uint32_t z = 8;
            if (sp.pitch) {
                scale[r] = scales[(r * 8 + g) * sp.pitch + at];
                if (p.zeros) z = zeros[(r * 8 + g) * sp.pitch + at] & 15u;
            } else {
                const int64_t i = group_row0 + int64_t(min(r * 8 + g, here - 1)) * groups + at;
                scale[r] = w4_scale<BF16>(p, i);
                if (p.zeros) z = p.zeros[i] & 15u;
            }
            less[r] = minus + z * 0x00010001u;
            less_up[r] = 0xD400D400u + z * 0x00100010u;  // -(64 + z)
        }
    };
    const int x_pitch = k * 2 + 64, vecs = k / 8;  // two tokens' rows fill all banks

    for (bool first = true;; first = false) {
        int count;
        if (p.pairs.experts) {
            if (warp == 0) {
                int n;
                const int next = list_pairs(p.pairs, expert, from, 8 * NT, list, n);
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
            count = min(8 * NT, p.pairs.pairs - from);
        }
        auto pair_at = [&](int i) { return p.pairs.experts ? list[i] : from + i; };
        auto x_row = [&](int i) { return p.x + int64_t(pair_at(min(i, count - 1)) / p.each) * p.ldx; };

        // What the first products wait for is asked for before the weights, which keep
        // the memory busy from then on: the first token's vectors of x, and scales,
        // kPerRow threads a row.
        const int my_vecs = HELD && expert >= 0 ? vecs : 0, my_row = int(threadIdx.x) / kPerRow;
        const int my_groups = first && my_row < here ? all_groups : 0;
        uint4 q[kW4Early];
        float v[2 * kW4Early];
        uint32_t z[2 * kW4Early];
        auto load_x = [&](int t, int j0) {
            const uint16_t *row = x_row(t);
#pragma unroll
            for (int e = 0; e < kW4Early; ++e)
                if (j0 + e * kThreads < my_vecs) q[e] = *reinterpret_cast<const uint4 *>(row + (j0 + e * kThreads) * 8);
        };
        auto store_x = [&](int t, int j0) {
            uint8_t *to = smem + sp.off_x + t * x_pitch;
#pragma unroll
            for (int e = 0; e < kW4Early; ++e)
                if (j0 + e * kThreads < my_vecs)
                    *reinterpret_cast<uint4 *>(to + w4_twist(unsigned(j0 + e * kThreads)) * 16) = w4_permuted(q[e]);
        };
        auto load_groups = [&](int i0) {
            const int64_t at = group_row0 + int64_t(my_row) * groups;
#pragma unroll
            for (int e = 0; e < 2 * kW4Early; ++e)
                if (i0 + e * kPerRow < my_groups) {
                    v[e] = w4_scale<BF16>(p, at + i0 + e * kPerRow);
                    if (p.zeros) z[e] = p.zeros[at + i0 + e * kPerRow];
                }
        };
        auto store_groups = [&](int i0) {
#pragma unroll
            for (int e = 0; e < 2 * kW4Early; ++e)
                if (i0 + e * kPerRow < my_groups) {
                    scales[my_row * sp.pitch + i0 + e * kPerRow] = v[e];
                    if (p.zeros) zeros[my_row * sp.pitch + i0 + e * kPerRow] = uint8_t(z[e]);
                }
        };
        const int lane_group = int(threadIdx.x) % kPerRow;
        load_x(0, int(threadIdx.x));
        load_groups(lane_group);
#pragma unroll
        for (int d = 0; d < kDepth; ++d) fetch(d, d);
        store_x(0, int(threadIdx.x));
        store_groups(lane_group);
        for (int i0 = lane_group + 2 * kW4Early * kPerRow; i0 < my_groups; i0 += 2 * kW4Early * kPerRow) {
            load_groups(i0);
            store_groups(i0);
        }
        if constexpr (HELD) {
            for (int t = 0; t < count; ++t)
                for (int j0 = int(threadIdx.x) + (t ? 0 : kW4Early * kThreads); j0 < my_vecs; j0 += kW4Early * kThreads) {
                    load_x(t, j0);
                    store_x(t, j0);
                }
        }
        __syncthreads();  // scales, zero points and x are there

        // Where this lane finds its vectors of x.
        const uint16_t *xs[NT];
        uint32_t xa[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (HELD)
                xa[t] = smem_addr(smem) + uint32_t(sp.off_x + min(t * 8 + g, count - 1) * x_pitch + chunk0 * 256);
            else
                xs[t] = x_row(t * 8 + g) + chunk0 * 128 + c * kWords * 8;
        }
        uint32_t x_at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x_at[i] = w4_twist(unsigned(i / kWords * 4 * kWords + c * kWords + i % kWords)) * 16;
        float total[R][NT][4] = {};
        for (int i0 = 0; i0 < n_chunks; i0 += kDepth) {
#pragma unroll
            for (int u = 0; u < kDepth; ++u) {
                const int i = i0 + u;
                if (i >= n_chunks) break;
                cp_async_wait<kDepth - 1>();
                __syncwarp();
#pragma unroll
                for (int s = 0; s < SUB; ++s) {
                    if (SUB > 1 && (chunk0 + i) * 128 + s * (128 / SUB) >= k) break;
                    float scale[2 * R];
                    uint32_t less[2 * R], less_up[2 * R], w[2 * R][kWords];
                    groups_of((chunk0 + i) * SUB + s, scale, less, less_up);
#pragma unroll
                    for (int r = 0; r < 2 * R; ++r) {
                        const int word = s * 4 * kWords + c * kWords;
                        const uint32_t a = ring + uint32_t(g * 64) + uint32_t((((word / 4) ^ twist) << 4) + word % 4 * 4) +
                                           uint32_t(u) * kChunkBytes + uint32_t(r * 512);
                        if constexpr (SUB == 1) {
                            const uint4 t = ld_shared_v4(a);
                            w[r][0] = t.x, w[r][1] = t.y, w[r][2] = t.z, w[r][3] = t.w;
                        } else if constexpr (SUB == 2) {
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[r][0]), "=r"(w[r][1]) : "r"(a) : "memory");
                        } else {
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[r][0]) : "r"(a) : "memory");
                        }
                    }
                    uint4 b[kWords][NT];
                    auto load_b = [&](int v) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if constexpr (HELD)
                                b[v][t] = ld_shared_v4(xa[t] + x_at[s * kWords + v] + uint32_t(u * 256));
                            else
                                b[v][t] = *reinterpret_cast<const uint4 *>(xs[t] + u * 128 + s * (128 / SUB) + v * 8);
                        }
                    };
                    constexpr int kEarly = R > 2 && kWords > 2 ? 2 : kWords;  // words of x on their way
#pragma unroll
                    for (int v = 0; v < kEarly; ++v) load_b(v);
                    float acc[R][NT][4];
#pragma unroll
                    for (int v = 0; v < kWords; ++v) {
                        if (v > 0 && v + kEarly - 1 < kWords) load_b(v + kEarly - 1);
                        if constexpr (!HELD) {
#pragma unroll
                            for (int t = 0; t < NT; ++t) b[v][t] = w4_permuted(b[v][t]);
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            uint32_t lo[4], hi[4];
                            spread<BF16>(w[2 * r][v], less[2 * r], less_up[2 * r], nib, lo);
                            spread<BF16>(w[2 * r + 1][v], less[2 * r + 1], less_up[2 * r + 1], nib, hi);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                if (v == 0)
                                    mma_first<BF16>(acc[r][t], lo[0], hi[0], lo[1], hi[1], b[v][t].x, b[v][t].y);
                                else
                                    mma_few<BF16>(acc[r][t], lo[0], hi[0], lo[1], hi[1], b[v][t].x, b[v][t].y);
                                mma_few<BF16>(acc[r][t], lo[2], hi[2], lo[3], hi[3], b[v][t].z, b[v][t].w);
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                total[r][t][e] = fmaf(acc[r][t][e], scale[2 * r + e / 2], total[r][t][e]);
                }
                __syncwarp();
                fetch(u, i + kDepth);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (HELD)
                    xa[t] += 256 * kDepth;
                else
                    xs[t] += 128 * kDepth;
            }
        }
        cp_async_wait<0>();
        __syncthreads();  // the rings are read
        // Not before: CTAs of the next launch would fill the SMs that finish first, unevenly
        // (4 of 32 experts of 2048 x 2048 for 4 tokens: 13.9 us, so 13.4).
        griddep_launch_dependents();
        float *part = reinterpret_cast<float *>(smem);  // [warps][16 R][8 NT + 1]
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    part[(warp * R * 16 + r * 16 + e / 2 * 8 + g) * (8 * NT + 1) + t * 8 + c * 2 + e % 2] = total[r][t][e];
        __syncthreads();
        for (int i = int(threadIdx.x); i < R * 16 * count; i += kThreads) {
            const int row = i % (R * 16), t = i / (R * 16);
            if (row >= here) continue;
            float sum = part[row * (8 * NT + 1) + t];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) sum += part[(w * R * 16 + row) * (8 * NT + 1) + t];
            const int64_t to = int64_t(pair_at(t)) * p.n + row0 + row;
            if (p.y_f32)
                static_cast<float *>(p.y)[to] = sum;
            else if (BF16)
                static_cast<__nv_bfloat16 *>(p.y)[to] = __float2bfloat16_rn(sum);
            else
                static_cast<__half *>(p.y)[to] = __float2half_rn(sum);
        }
        if (!p.pairs.experts || from >= p.pairs.pairs) return;
        __syncthreads();  // the sums and the list are read
    }
}

static bool w4_staged(const W4 &p, int r) { return 16 * r * (p.groups | 1) * (p.zeros ? 5 : 4) <= kW4Scales; }

template <bool BF16, int SUB, int WARPS, int NT, int R, bool HELD>
static int w4_launch(const W4 &p, int tokens, const Device &d, cudaStream_t s)
{
    const int64_t blocks = (p.n + 16 * R - 1) / (16 * R);
    const int slots = p.pairs.experts ? slots_of(p.pairs) : 1;
    const int passes = p.pairs.experts ? 1 : (p.pairs.pairs + 8 * NT - 1) / (8 * NT);
    if (blocks > 2147483647 || slots > 65535 || passes > 65535) return kErrInvalidArg;
    constexpr int ring = W4Ring<WARPS, NT, R>::kBytes;
    W4Space sp{};
    const int64_t room = 16 * R * (p.groups | 1), zeros = p.zeros ? room : 0;
    const bool staged = w4_staged(p, R);
    sp.pitch = staged ? int(p.groups | 1) : 0;
    sp.off_zeros = ring + (staged ? int(room * 4) : 0);
    sp.off_x = sp.off_zeros + (staged ? int(zeros) : 0);
    sp.total = sp.off_x + (HELD ? int(tokens * (p.k * 2 + 64)) : 0);
    static std::once_flag once[64];
    bool ok = true;
    auto set = [&] {
        const int64_t most = ring + kW4Scales + (HELD ? kW4Held : 0);
        ok = cudaFuncSetAttribute(w4_kernel<BF16, SUB, WARPS, NT, R, HELD>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most)) ==
             cudaSuccess;
    };
    if (d.ordinal < 64)
        std::call_once(once[d.ordinal], set);
    else
        set();
    if (!ok) {
        cudaGetLastError();
        return kErrCuda;
    }
    return launch(w4_kernel<BF16, SUB, WARPS, NT, R, HELD>, dim3(unsigned(blocks), unsigned(slots), unsigned(passes)),
                  dim3(32 * WARPS), size_t(sp.total), s, 1, p, sp);
}

template <bool BF16, int SUB>
static int w4_shape(const W4 &p, const Device &d, cudaStream_t s)
{
    // tokens that one matrix can have, evenly spread
    const int pairs = p.pairs.pairs, tokens = p.pairs.experts ? (pairs + p.pairs.num_experts - 1) / p.pairs.num_experts : pairs;
    if (tokens > 16) {
        // One CTA an SM, each reading all of x from L2.  64 rows halve that and take 1.65
        // times as long as 32, so they pay where they save rounds: 32 tokens, 16384 x 8192
        // 54.7 us against 63.5, 9728 x 4096 17.1 against 20.3, 4096 x 4096 17.4 against 10.6.
        // With 64 rows the kernel takes 255 registers and spills 236 bytes in bf16, 332 in fp16
        // (groups of 128).
        const int64_t each = p.pairs.experts ? p.pairs.num_experts : (pairs + 31) / 32;
        const int64_t rounds2 = ((p.n + 31) / 32 * each + d.sms - 1) / d.sms, rounds4 = ((p.n + 63) / 64 * each + d.sms - 1) / d.sms;
        return 1.65 * double(rounds4) < double(rounds2) && w4_staged(p, 4) ? w4_launch<BF16, SUB, 8, 4, 4, false>(p, 32, d, s)
                                                                          : w4_launch<BF16, SUB, 8, 4, 2, false>(p, 32, d, s);
    }
    // With CTAs enough four of them with four warps share an SM, otherwise two with eight
    // that share out k further: 16384 x 8192 20.7 us against 23.4, 4096 x 4096 5.7 against
    // 5.6; 12 tokens, 5001 x 4096 13.2 against 11.0.
    // Scales of more than 128 groups a row take longer to fetch with four warps, and
    // leave room for fewer CTAs (groups of 32 at 8192: 58 us against 39).
    const bool many = (p.n + 31) / 32 * (p.pairs.experts ? slots_of(p.pairs) : 1) >= 2 * d.sms && p.groups <= 128;
    if (tokens > 8) return many ? w4_launch<BF16, SUB, 4, 2, 2, false>(p, 16, d, s) : w4_launch<BF16, SUB, 8, 2, 2, false>(p, 16, d, s);
    const int most = pairs < 8 ? pairs : 8;
    if (most * (p.k * 2 + 64) <= kW4Held)
        return many ? w4_launch<BF16, SUB, 4, 1, 2, true>(p, most, d, s) : w4_launch<BF16, SUB, 8, 1, 2, true>(p, most, d, s);
    return many ? w4_launch<BF16, SUB, 4, 1, 2, false>(p, most, d, s) : w4_launch<BF16, SUB, 8, 1, 2, false>(p, most, d, s);
}

template <bool BF16>
static int w4(const W4 &p, const Device &d, cudaStream_t s)
{
    if (p.group % 128 == 0) return w4_shape<BF16, 1>(p, d, s);
    if (p.group % 64 == 0) return w4_shape<BF16, 2>(p, d, s);
    return w4_shape<BF16, 4>(p, d, s);
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
    p.y = y;
    p.n = n;
    p.k = k;
    p.group = group;
    p.groups = k / group;
    p.pairs = Pairs{experts, int(pairs), int(num_experts)};
    p.each = int(each);
    p.scales_f32 = scale_dtype == kF32;
    p.y_f32 = y_dtype == kF32;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == kBF16 ? w4<true>(p, d, s) : w4<false>(p, d, s);
}
