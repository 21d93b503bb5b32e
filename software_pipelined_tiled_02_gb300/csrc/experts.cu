// experts.cu -- the gated feed-forward blocks of a mixture of experts, forward and
// backward, for GB300 (sm_103a), and their C ABI.
//
// Every pair of a token and an expert is a row, in expert order (experts.cuh):
//   g = x Wg_e^T,  u = x Wu_e^T,  h = act(g) u,  y_t = sum over t's pairs of w h Wd_e^T
//   dh = dy Wd_e,  dw = <dh, h>,  dg = w dh u act'(g),  du = w dh act(g)
//   dx_t = sum over t's pairs of dg Wg_e + du Wu_e
//   dWg_e = dg^T x,  dWu_e = du^T x,  dWd_e = dy^T (w h)   over e's rows
//
// The products are those of ffn.cu with a third coordinate, the expert, and run
// through the same pipeline: a ring of slots of 64 reduction elements filled by
// TMA, tcgen05.mma on CTA pairs with 256 rows a tile, and eight warps that drain
// one of two tensor-memory accumulators while the next tile's MMAs fill the other.
//   Up    g, u and h (256 columns: the same 128 of Wg and of Wu)
//   Down  h Wd^T in fp32, which the combining kernel weighs and adds
//   Dh    dg, du, w h and dw's partial sums over a tile's columns
//   Dx    dg Wg + du Wu in fp32
//   Dw    all three weight gradients of all experts as one list of tiles; the
//         reduction runs over the expert's rows
// How many rows an expert has is known on the GPU alone: the placing kernel leaves
// a list of row tiles there, every CTA pair reads its length, and the host's grid
// is one pair per two SMs.  Nothing waits for the host.
//
// What bounds it, cold and at full clocks: 8192 tokens, 4 of 32 experts of 4096 x 2048
// bf16: Up 690 us, Down 355 (1.6 PFLOP/s, with the rows that fill up the last tile of
// each expert 1.8).  Backward, 6 of 64 experts of 2048 x 1408: Dh 284 us, half of the
// cycles with the tensor pipe active (its epilogue moves six tensors), Dx 380, Dw 620
// (12 blocks a tile: a tile's end takes about as long as its sums).  A whole forward
// pass with gathering and combining takes 1.24 to 1.39 ms, a backward pass of the second
// size 1.49 to 1.67, the longer ones under the power cap.  48 tokens, 4 of 32 experts
// of 4096 x 1536: 201 to 204 us for 1.2 GB of weights, 5.9 TB/s.
//
// Down's and Dx's results stay fp32 until they are added: a third rounding to 16
// bits would cost more than the two that the operands of Down and Dx need.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>

#include "experts.cuh"
#include "ffn.cuh"
#include "host.h"
#include "layout.h"
#include "ptx.cuh"
#include "tgemm.h"
#include "watchdog.cuh"

namespace tg {

constexpr uint32_t kBox = 32 * 64;  // a box of an epilogue warp: 32 rows of 64 bytes
[[maybe_unused]] constexpr int kAccStride = 256;  // tensor-memory columns between the two accumulators

// A product's shared memory: the ring's A and B slots, the epilogue warps' boxes
// (Dh: three that come in and go out), the barriers.
template <int PROD>
struct ExpertLayout {
    // In Dh each box that came in goes out again, which leaves room for a fifth slot:
    // with boxes of their own and four slots 297 us (8192 tokens, 6 of 64 experts of
    // 2048 x 1408), so 284; sixteen epilogue warps with four slots took 306.
    static constexpr int kStages = PROD == kDown || PROD == kDx ? 6 : 5;
    static constexpr int kBoxes = PROD == kDh ? 3 : PROD == kUp ? 3 : PROD == kDw ? 4 : 2;  // per epilogue warp
    static constexpr uint32_t kOffB = kStages * kSlot, kOffC = 2 * kStages * kSlot;
    static constexpr uint32_t kOffBar = kOffC + kBoxes * kEpiWarps * kBox;
    static constexpr int kBars = 2 * kStages + 6 + kEpiWarps;
    static constexpr uint32_t kTotal = kOffBar + 8 * kBars + 16 + kSmemAlign;
};

struct ExpertParams {  // 64-byte aligned through its CUtensorMap members
    // By index: Up reads B by CTA rank (gate, up) and stores h, g, u; Dh reads g, u,
    // h and stores dg, du, w h; Dx reads A and B by K segment; Dw reads and stores
    // by problem.
    CUtensorMap tmA[3], tmB[3], tmC[3], tmIn[3];
    void *out[3];             // Up: h, g, u, for rows that share a box with another expert's
    int m[3], n[3];           // Dw: rows and columns of each problem's output; otherwise n[0]
    int tiles_m[3], tiles_n[3];
    int first[4];             // Dw: first tile of each problem among an expert's, then their number
    int problems, experts;
    int bn, tile_cols, num_kb, seg_kb, group_m;
    uint32_t idesc, stage_tx;
    int act, save;
    int beside;               // Dw: see ExpertJob
    const RowTile *table;
    const int *tiles, *padded, *pair_of;
    const float *weights;     // Dh
    float *parts;             // Dh: [2 tiles_n][padded rows]
    int64_t part_stride;
    unsigned long long watchdog_ns;
    int *status;
    int debug_stall;
};

// What one tile is: its output block, its expert, its rows (or, for Dw, the
// reduction's).
struct ExpertTile {
    int prob, mb, nb;
    RowTile rows;
    int num_kb;
};

template <int PROD>
__device__ __forceinline__ ExpertTile expert_tile(const ExpertParams &p, int t, int row_tiles)
{
    ExpertTile w;
    w.prob = 0;
    w.num_kb = p.num_kb;
    if constexpr (PROD == kDw) {
        const int e = t / p.first[p.problems];
        int r = t - e * p.first[p.problems];
        while (w.prob + 1 < p.problems && r >= p.first[w.prob + 1]) ++w.prob;
        r -= p.first[w.prob];
        w.mb = r % p.tiles_m[w.prob];
        w.nb = r / p.tiles_m[w.prob];
        const int first = p.padded[e], rows = p.padded[e + 1] - first;
        w.rows = RowTile{e, first, first, rows};
        w.num_kb = (rows + kBlockK - 1) / kBlockK;
    } else {
        const int per_group = p.group_m * p.tiles_n[0];
        const int grp = t / per_group, first_m = grp * p.group_m;
        const int gm = min(p.group_m, row_tiles - first_m);
        const int r = t - grp * per_group;
        w.mb = first_m + r % gm;
        w.nb = r / gm;
        const int4 q = __ldg(reinterpret_cast<const int4 *>(p.table + w.mb));
        w.rows = RowTile{q.x, q.y, q.z, q.w};
    }
    return w;
}

template <int PROD, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) experts_gemm_kernel(const __grid_constant__ ExpertParams p)
{
    constexpr bool A_MN = PROD == kDw, B_MN = PROD == kDh || PROD == kDx || PROD == kDw;
    using L = ExpertLayout<PROD>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = (kSmemAlign - (raw & (kSmemAlign - 1))) & (kSmemAlign - 1);
    uint8_t *smem = smem_raw + pad;
    const uint32_t sA = raw + pad, sB = sA + L::kOffB, sC = sA + L::kOffC, bars = sA + L::kOffBar;
    auto full = [&](int s) { return bars + 8u * uint32_t(s); };
    auto empty = [&](int s) { return bars + 8u * uint32_t(kStages + s); };
    auto acc_full = [&](int a) { return bars + 8u * uint32_t(2 * kStages + a); };
    auto acc_empty = [&](int a) { return bars + 8u * uint32_t(2 * kStages + 2 + a); };
    const uint32_t drain = bars + 8u * uint32_t(2 * kStages + 4);
    const uint32_t stall = bars + 8u * uint32_t(2 * kStages + 5);
    auto box_in = [&](int w) { return bars + 8u * uint32_t(2 * kStages + 6 + w); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffBar + 8 * L::kBars);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32;
    const uint32_t rank = cluster_ctarank();
    const int pair = int(blockIdx.x >> 1), pairs = int(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full(a), 1);
            mbar_init(acc_empty(a), 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        mbar_init(stall, 1);
        for (int w = 0; w < kEpiWarps; ++w) mbar_init(box_in(w), 1);
        *abort = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tmA[0]);
        prefetch_tmap(&p.tmB[PROD == kUp ? rank : 0]);
        prefetch_tmap(&p.tmC[0]);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(tmem_slot), kTmemColsMax);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (PROD != kDw || !p.beside) griddep_wait();
    griddep_launch_dependents();
    const int row_tiles = PROD == kDw ? 0 : *p.tiles;
    const int tiles = PROD == kDw ? p.experts * p.first[p.problems] : row_tiles * p.tiles_n[0];

    if (warp == 0 || warp == kProducerBWarp) {
        // Producers: one lane each, up to kStages slots ahead.  Each CTA loads its 128
        // rows of A and its half of B's columns; both complete the even CTA's full[s].
        if (lane == 0) {
            const uint32_t full_leader = map_to_rank(full(0), 0);
            const int b_rows = p.bn / 2;
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {  // a wait that fails ends the loop
                const ExpertTile w = expert_tile<PROD>(p, t, row_tiles);
                const int a0 = (PROD == kDw ? w.mb * 256 : PROD == kDown ? w.rows.row : w.rows.padded) + int(rank) * 128;
                const int n0 = PROD == kUp ? w.nb * p.tile_cols : w.nb * p.bn + int(rank) * b_rows;
                for (int kb = 0; kb < w.num_kb; ++kb) {
                    if (!mbar_try_wait(empty(s), ph ^ 1u) && !wait_bar(empty(s), ph ^ 1u, p, abort, 0, issued)) {
                        ok = false;
                        break;
                    }
                    const int seg = PROD == kDx && kb >= p.seg_kb ? 1 : 0;
                    const int k = (kb - (seg ? p.seg_kb : 0)) * kBlockK;
                    const int ia = PROD == kDw ? w.prob : seg;
                    const int ib = PROD == kUp ? int(rank) : ia;
                    if (!check(s < kStages && w.rows.expert < p.experts && w.nb < p.tiles_n[w.prob] && n0 % 8 == 0, p, abort, 0,
                               issued)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full_leader + 8u * uint32_t(s);
                    if (warp == 0) {
                        const uint32_t dst = sA + uint32_t(s) * kSlot;
                        if (rank == 0) mbar_arrive_expect_tx(full(s), p.stage_tx);
                        if constexpr (A_MN) {
                            tma_load_2d_pair(dst, &p.tmA[ia], a0, w.rows.padded + k, bar);
                            tma_load_2d_pair(dst + kPanel, &p.tmA[ia], a0 + 64, w.rows.padded + k, bar);
                        } else {
                            tma_load_2d_pair(dst, &p.tmA[ia], k, a0, bar);
                        }
                    } else {
                        const uint32_t dst = sB + uint32_t(s) * kSlot;
                        if constexpr (PROD == kDw) {
                            tma_load_2d_pair(dst, &p.tmB[ib], n0, w.rows.padded + k, bar);
                            if (b_rows > 64) tma_load_2d_pair(dst + kPanel, &p.tmB[ib], n0 + 64, w.rows.padded + k, bar);
                        } else if constexpr (B_MN) {
                            tma_load_3d_pair(dst, &p.tmB[ib], n0, k, w.rows.expert, bar);
                            if (b_rows > 64) tma_load_3d_pair(dst + kPanel, &p.tmB[ib], n0 + 64, k, w.rows.expert, bar);
                        } else {
                            tma_load_3d_pair(dst, &p.tmB[ib], k, n0, w.rows.expert, bar);
                        }
                    }
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // MMA issuer (even CTA): the converged warp, one elected lane issues.
        if (rank == 0) {
            const uint64_t ad0 = ffn_desc(sA, A_MN), bd0 = ffn_desc(sB, B_MN);
            // 16 reduction elements further on, in 16-byte units (ffn.cu)
            constexpr uint64_t a_step = A_MN ? 2048 >> 4 : 32 >> 4, b_step = B_MN ? 2048 >> 4 : 32 >> 4;
            int s = 0, a = 0, it = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            if (p.debug_stall) ok = warp_wait(stall, 0, p, abort, 1, 0);  // test hook: nothing arrives
            for (int t = pair; ok && t < tiles; t += pairs) {
                int num_kb = p.num_kb, rows = 0;
                if constexpr (PROD == kDw) {
                    const ExpertTile w = expert_tile<PROD>(p, t, row_tiles);
                    num_kb = w.num_kb;
                    rows = w.rows.rows;
                }
                if (!warp_wait(acc_empty(a), aph ^ 1u, p, abort, 1, it)) break;
                tc_fence_after();
                const uint32_t d = tmem + uint32_t(a * kAccStride);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!warp_wait(full(s), ph, p, abort, 1, it)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = ad0 + uint64_t(s) * (kSlot >> 4), bd = bd0 + uint64_t(s) * (kSlot >> 4);
                    // Dw: an expert's rows fill a multiple of 32; the block's others are the next expert's
                    const int steps = PROD == kDw ? min(kBlockK / 16, (rows - kb * kBlockK) / 16) : kBlockK / 16;
#pragma unroll
                    for (int kk = 0; kk < kBlockK / 16; ++kk)
                        if (PROD != kDw || kk < steps)
                            mma_f16_pair(d, ad + uint64_t(kk) * a_step, bd + uint64_t(kk) * b_step, p.idesc,
                                         kk || kb ? 1u : 0u);
                    mma_commit_pair_elect(empty(s), uint16_t(0x3));
                    __syncwarp();
                    ++it;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair_elect(acc_full(a), uint16_t(0x3));
                __syncwarp();
                a ^= 1;
                if (a == 0) aph ^= 1u;
            }
            if (lane == 0) {  // every MMA issued has to finish before TMEM is freed
                mma_commit_pair(drain, uint16_t(0x1));
                wait_bar(drain, 0, p, abort, 1, it, false);
            }
            __syncwarp();
        }
    } else {
        // Epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31, lane = output row;
        // the two warps of a quarter take alternate chunks of 32 columns.
        const int q = warp & 3, sub = (warp - 2) >> 2;
        const uint32_t lane_base = uint32_t(q * 32) << 16;
        const uint32_t my_bufs = sC + uint32_t(L::kBoxes * (warp - 2)) * kBox;
        uint32_t boxes = 0, aph = 0;
        int a = 0, done = 0;
        // 16 words of this lane's row to box k, swizzled as the tensor maps say.
        auto stage = [&](int k, const uint32_t *w) {
            const uint32_t at = my_bufs + uint32_t(k) * kBox + uint32_t(lane) * 64u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                st_shared_v4(at + (uint32_t(j ^ ((lane >> 1) & 3)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        };
        // Two neighbouring boxes with one fence (Down, Dx, Dw); `both`: the second has columns.
        [[maybe_unused]] auto put_two = [&](const CUtensorMap *map, int col, int width, int row, int z, bool both, const uint32_t *w) {
            const int k = PROD == kDw ? int(boxes & 1u) * 2 : 0;
            if (lane == 0) bulk_wait_read<PROD == kDw ? 1 : 0>();
            __syncwarp();
            stage(k, w);
            if (both) stage(k + 1, w + 16);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                for (int i = 0; i < (both ? 2 : 1); ++i) {
                    const uint32_t from = my_bufs + uint32_t(k + i) * kBox;
                    if constexpr (PROD == kDw)
                        tma_store_3d(map, col + i * width, row, z, from);
                    else
                        tma_store_2d(map, col + i * width, row, from);
                }
                bulk_commit();
            }
            ++boxes;
        };
        // `count` boxes of the same place in as many outputs, with one fence (Up).
        [[maybe_unused]] auto put_all = [&](int count, int col, int row, const uint32_t (&w)[3][16]) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < count) stage(i, w[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                for (int i = 0; i < count; ++i) tma_store_2d(&p.tmC[i], col, row, my_bufs + uint32_t(i) * kBox);
                bulk_commit();
            }
        };
        [[maybe_unused]] auto packed = [&](const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack2(v[2 * e], v[2 * e + 1], BF16);
        };
        auto read = [&](uint32_t col, float (&v)[32]) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tmem + lane_base + col, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
        };
        const int first_row = int(rank) * 128 + q * 32;  // of this warp, in a tile
        // Dh: this warp's boxes of g, u and h for its next chunk; what it stored from them
        // has been read by then.
        [[maybe_unused]] const uint32_t in_bar = box_in(warp - 2);
        [[maybe_unused]] uint32_t in_ph = 0;
        [[maybe_unused]] bool coming = false;
        [[maybe_unused]] auto fetch = [&](const ExpertTile &w, int c) -> bool {
            const int col = w.nb * p.tile_cols + c * 32;
            if (c * 32 >= p.tile_cols || first_row >= w.rows.rows || col >= p.n[0]) return false;
            __syncwarp();  // every lane has read the boxes
            if (lane == 0) {
                bulk_wait_read<0>();
                mbar_arrive_expect_tx(in_bar, 3 * kBox);
                for (int i = 0; i < 3; ++i) tma_load_2d(my_bufs + uint32_t(i) * kBox, &p.tmIn[i], col, w.rows.row + first_row, in_bar);
            }
            coming = true;
            return true;
        };
        if constexpr (PROD == kDh) {
            if (pair < tiles) fetch(expert_tile<PROD>(p, pair, row_tiles), sub);
        }
        for (int t = pair; t < tiles; t += pairs, ++done) {
            const ExpertTile w = expert_tile<PROD>(p, t, row_tiles);
            const int n0 = w.nb * p.tile_cols, n = p.n[w.prob];
            const int rows = PROD == kDw ? p.m[w.prob] - w.mb * 256 : w.rows.rows;  // of the tile's output
            const bool mine = first_row + lane < rows;
            [[maybe_unused]] float weight = 0.f, dot = 0.f;
            if constexpr (PROD == kDh) {
                if (mine) weight = p.weights[p.pair_of[w.rows.padded + first_row + lane]];
            }
            if (!warp_wait(acc_full(a), aph, p, abort, 2, done)) break;
            tc_fence_after();
            const uint32_t acc = uint32_t(a * kAccStride);
            constexpr int kWide = PROD == kDw ? 64 : 32;  // columns of a chunk
            for (int c = sub; c * kWide < p.tile_cols && first_row < rows && n0 + c * kWide < n; c += 2) {
                const int col = n0 + c * kWide;
                if (!check(int(acc) + (PROD == kUp ? p.tile_cols : 0) + c * kWide + 32 <= kTmemColsMax && col % 8 == 0, p, abort,
                           2, done))
                    break;
                if constexpr (PROD == kUp) {
                    uint32_t o[3][16];
                    float g[32], u[32];
                    read(acc + uint32_t(c * 32), g);
                    read(acc + uint32_t(p.tile_cols + c * 32), u);
                    if (p.save) {
                        packed(g, o[1]);
                        packed(u, o[2]);
                    }
                    auto gate = [&](auto act_c) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            F2 act, slope;
                            activate<decltype(act_c)::value>(f2(g[e], g[e + 1]), act, slope);
                            o[0][e / 2] = pack2(act * f2(u[e], u[e + 1]), BF16);
                        }
                    };
                    if (p.act == kSilu)
                        gate(std::integral_constant<int, kSilu>{});
                    else if (p.act == kGelu)
                        gate(std::integral_constant<int, kGelu>{});
                    else
                        gate(std::integral_constant<int, kRelu>{});
                    const int count = p.save ? 3 : 1;
                    if (first_row + 32 <= rows) {
                        put_all(count, col, w.rows.row + first_row, o);
                    } else if (mine) {  // the box reaches into the next expert's rows: each lane stores its own
                        for (int i = 0; i < count; ++i) {
                            uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out[i]) +
                                                                  int64_t(w.rows.row + first_row + lane) * n + col);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (col + 8 * j < n) {
                                    const uint32_t *v = i == 0 ? o[0] : i == 1 ? o[1] : o[2];
                                    to[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                                }
                        }
                    }
                } else if constexpr (PROD == kDh) {
                    // This lane's row of g, u and h, 16 columns at a time; dg, du and w h take their
                    // places.
                    if (!warp_wait(in_bar, in_ph, p, abort, 2, done)) break;
                    in_ph ^= 1u;
                    coming = false;
                    const F2 scale = f2(weight);
                    F2 sum = f2(0.f);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t dh[16];
                        tmem_ld_32x32b_x16(tmem + lane_base + acc + uint32_t(c * 32 + half * 16), dh);
                        const uint32_t at = my_bufs + uint32_t(lane) * 64u;
                        auto place = [&](int i, int j) {  // words 4 j .. of box i's half row, swizzled as the maps say
                            return at + uint32_t(i) * kBox + (uint32_t((half * 2 + j) ^ ((lane >> 1) & 3)) << 4);
                        };
                        uint32_t io[3][8];
#pragma unroll
                        for (int i = 0; i < 3; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint4 v = ld_shared_v4(place(i, j));
                                io[i][4 * j] = v.x, io[i][4 * j + 1] = v.y, io[i][4 * j + 2] = v.z, io[i][4 * j + 3] = v.w;
                            }
                        tmem_wait_ld();
                        auto ungate = [&](auto act_c) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 g2 = unpack2(io[0][j], BF16), u2 = unpack2(io[1][j], BF16), h2 = unpack2(io[2][j], BF16);
                                const F2 d = f2(__uint_as_float(dh[2 * j]), __uint_as_float(dh[2 * j + 1]));
                                const F2 h = f2(h2.x, h2.y), dw = d * scale;
                                sum = fma2(d, h, sum);
                                F2 act, slope;
                                activate<decltype(act_c)::value>(f2(g2.x, g2.y), act, slope);
                                // rows behind the expert's last hold what the next one's computes: zero
                                io[0][j] = mine ? pack2(dw * f2(u2.x, u2.y) * slope, BF16) : 0u;
                                io[1][j] = mine ? pack2(dw * act, BF16) : 0u;
                                io[2][j] = mine ? pack2(h * scale, BF16) : 0u;
                            }
                        };
                        if (p.act == kSilu)
                            ungate(std::integral_constant<int, kSilu>{});
                        else if (p.act == kGelu)
                            ungate(std::integral_constant<int, kGelu>{});
                        else
                            ungate(std::integral_constant<int, kRelu>{});
#pragma unroll
                        for (int i = 0; i < 3; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                st_shared_v4(place(i, j), io[i][4 * j], io[i][4 * j + 1], io[i][4 * j + 2], io[i][4 * j + 3]);
                    }
                    dot += sum2(sum);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        for (int i = 0; i < 3; ++i)
                            tma_store_2d(&p.tmC[i], col, w.rows.padded + first_row, my_bufs + uint32_t(i) * kBox);
                        bulk_commit();
                    }
                    if (!fetch(w, c + 2) && t + pairs < tiles) fetch(expert_tile<PROD>(p, t + pairs, row_tiles), sub);
                } else {
                    float v[32];
                    read(acc + uint32_t(c * kWide), v);
                    if constexpr (PROD == kDw) {
                        const bool both = (c * 2 + 1) * 32 < p.tile_cols && col + 32 < n;
                        uint32_t o[2][16];
                        packed(v, o[0]);
                        if (both) {
                            read(acc + uint32_t(c * kWide + 32), v);
                            packed(v, o[1]);
                        }
                        if (w.num_kb == 0) {  // an expert without rows
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[0][e] = o[1][e] = 0u;
                        }
                        put_two(&p.tmC[w.prob], col, 32, w.mb * 256 + first_row, w.rows.expert, both, o[0]);
                    } else {
                        uint32_t o[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(mine ? v[e] : 0.f);
                        put_two(&p.tmC[0], col, 16, w.rows.padded + first_row, 0, col + 16 < n, o);
                    }
                }
            }
            if constexpr (PROD == kDh) {
                if (first_row < rows) p.parts[int64_t(2 * w.nb + sub) * p.part_stride + w.rows.padded + first_row + lane] = dot;
                // no chunk of this tile was this warp's: the next tile's boxes were not asked for
                if (!coming && t + pairs < tiles) fetch(expert_tile<PROD>(p, t + pairs, row_tiles), sub);
            }
            // All TMEM reads of accumulator a are done: hand it back.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(acc_empty(a), 0));
            a ^= 1;
            if (a == 0) aph ^= 1u;
        }
        if constexpr (PROD == kDh) {
            if (coming) warp_wait(in_bar, in_ph, p, abort, 2, done, false);  // boxes on their way land before the CTA exits
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (*abort && threadIdx.x == 0) {
        // Loads in flight land before the CTA may exit; no barrier is known to
        // complete for them (tgemm.cu), so they get 2 ms.
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 2000000ull) {
        }
    }
    if (PROD == kDw && p.beside) griddep_wait();
    __syncwarp();
    cluster_sync();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem, kTmemColsMax);
    }
}

// ---------------------------------------------------------------- host side

typedef void (*ExpertKernel)(const ExpertParams);
static const ExpertKernel kExpertKernels[2][5] = {  // by type (fp16, bf16) and product
    {experts_gemm_kernel<kUp, false>, experts_gemm_kernel<kDown, false>, experts_gemm_kernel<kDh, false>,
     experts_gemm_kernel<kDx, false>, experts_gemm_kernel<kDw, false>},
    {experts_gemm_kernel<kUp, true>, experts_gemm_kernel<kDown, true>, experts_gemm_kernel<kDh, true>,
     experts_gemm_kernel<kDx, true>, experts_gemm_kernel<kDw, true>}};
static const uint32_t kExpertSmem[5] = {ExpertLayout<kUp>::kTotal, ExpertLayout<kDown>::kTotal, ExpertLayout<kDh>::kTotal,
                                        ExpertLayout<kDx>::kTotal, ExpertLayout<kDw>::kTotal};

// Once per device: the kernels' shared-memory ceiling.
static int experts_setup(const Device &d)
{
    static std::mutex mu;
    static bool known[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (d.ordinal < 64 && known[d.ordinal]) return kOk;
    for (int i = 0; i < 5; ++i) {
        if (int(kExpertSmem[i]) > d.smem_limit) return kErrSmemBudget;
        for (const auto &type : kExpertKernels) {
            if (cudaFuncSetAttribute(type[i], cudaFuncAttributeMaxDynamicSharedMemorySize, int(kExpertSmem[i])) != cudaSuccess) {
                cudaGetLastError();
                return kErrCuda;
            }
        }
    }
    if (d.ordinal < 64) known[d.ordinal] = true;
    return kOk;
}

// One matrix for each expert: `rows` x `cols`, `ld` from row to row, `es` from
// expert to expert.
struct Stack {
    const void *p;
    int64_t rows, cols, ld, es;
};

struct ExpertJob {
    int prod, problems;
    int64_t k;       // reduction length of one segment; Dw: unused
    int na, nb, nc;
    Mat A[3];
    Stack B[3];      // Dw: plain matrices (rows: the padded ones)
    Stack C[3];      // Dw: the gradients; otherwise plain matrices
    Mat in[3];       // Dh
    // Dw launched right after Dx: it reads nothing that Dx writes, and Dx lets it start
    // only once Dh has finished, so it fills the SMs that Dx leaves, and waits for Dx at
    // its own end.
    bool beside;
    bool shared;  // Dx and Dw of one call
    const float *weights;
    float *parts;
    int64_t part_stride;
};

// Columns of a tile: as ffn.cu's tile_width, with the row tiles that evenly spread
// pairs would have.  Dx and Dw beside each other weigh the SMs that they take from
// one another.
static int expert_tile_width(const tgemm_ffn_s *f, const ExpertJob &j, const ExpertSizes &z, int num_kb)
{
    const double used = double(z.experts < z.pairs ? z.experts : z.pairs), each = double(z.pairs) / used;
    const double row_tiles = used * (each <= kRowTile / 2 ? 1.0 : each / kRowTile + 0.5);
    int best = 256;
    double best_cost = 0.0;
    for (int bn = 256; bn >= 64; bn -= 32) {
        if (j.prod == kUp && bn % 64) continue;  // whole 32-column chunks of both projections
        const int cols = j.prod == kUp ? bn / 2 : bn;
        double tiles = 0.0;
        for (int i = 0; i < j.problems; ++i) {
            const double across = double((j.C[i].cols + cols - 1) / cols);
            tiles += j.prod == kDw ? double(z.experts) * double((j.C[i].rows + 255) / 256) * across : row_tiles * across;
        }
        const double blocks = j.prod == kDw ? each / kBlockK + 0.5 : double(num_kb);
        const double beside = 260.0 + 1.7 * bn > 630.0 ? 260.0 + 1.7 * bn : 630.0;
        const double tile = (j.shared ? beside : 580.0) * blocks + 2000.0 + 18.0 * bn;
        const double waves = tiles / f->pairs;
        const double cost = (waves < 1.0 ? 1.0 : waves + 0.5) * tile + (j.shared ? kShare * waves * tile : 0.0);
        if (bn == 256 || cost < best_cost) {
            best = bn;
            best_cost = cost;
        }
    }
    return best;
}

static int expert_product(tgemm_ffn_s *f, const ExpertJob &j, const ExpertSizes &z, const Placed &at, cudaStream_t s)
{
    ExpertParams p;
    std::memset(&p, 0, sizeof(p));
    const bool a_mn = j.prod == kDw, b_mn = j.prod == kDh || j.prod == kDx || j.prod == kDw;
    p.problems = j.problems;
    p.experts = int(z.experts);
    p.seg_kb = int((j.k + kBlockK - 1) / kBlockK);
    p.num_kb = j.prod == kDx ? 2 * p.seg_kb : p.seg_kb;
    p.bn = expert_tile_width(f, j, z, p.num_kb);
    p.tile_cols = j.prod == kUp ? p.bn / 2 : p.bn;
    p.group_m = 8;
    p.save = j.nc == 3 && j.prod == kUp;
    int64_t total = 0;
    for (int i = 0; i < j.problems; ++i) {
        p.m[i] = int(j.C[i].rows);
        p.n[i] = int(j.C[i].cols);
        p.tiles_m[i] = int((j.C[i].rows + 255) / 256);
        p.tiles_n[i] = int((j.C[i].cols + p.tile_cols - 1) / p.tile_cols);
        p.first[i] = int(total);
        total += int64_t(p.tiles_m[i]) * p.tiles_n[i];
    }
    p.first[j.problems] = int(total);
    const int64_t most = j.prod == kDw ? total * z.experts : z.row_tiles * p.tiles_n[0];
    if (total > (int64_t(1) << 30) || most > (int64_t(1) << 30)) return kErrInvalidArg;
    const int b_rows = p.bn / 2;
    int rc = kOk;
    for (int i = 0; i < j.na && rc == kOk; ++i) {
        const uint64_t pitch = uint64_t(j.A[i].ld) * 2;
        rc = encode_2d(&p.tmA[i], f->dtype, j.A[i].p, uint64_t(j.A[i].cols), uint64_t(j.A[i].rows), pitch, 64, a_mn ? 64u : 128u,
                       CU_TENSOR_MAP_SWIZZLE_128B, operand_promotion(pitch));
    }
    for (int i = 0; i < j.nb && rc == kOk; ++i) {
        const Stack &b = j.B[i];
        const uint64_t pitch = uint64_t(b.ld) * 2;
        if (j.prod == kDw)
            rc = encode_2d(&p.tmB[i], f->dtype, b.p, uint64_t(b.cols), uint64_t(b.rows), pitch, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B,
                           operand_promotion(pitch));
        else
            rc = encode_3d(&p.tmB[i], f->dtype, b.p, uint64_t(b.cols), uint64_t(b.rows), uint64_t(z.experts), pitch,
                           uint64_t(b.es) * 2, 64, b_mn ? 64u : uint32_t(b_rows), CU_TENSOR_MAP_SWIZZLE_128B,
                           operand_promotion(pitch));
    }
    for (int i = 0; i < j.nc && rc == kOk; ++i) {
        const Stack &c = j.C[i];
        if (j.prod == kDw)
            rc = encode_3d(&p.tmC[i], f->dtype, c.p, uint64_t(c.cols), uint64_t(c.rows), uint64_t(z.experts), uint64_t(c.ld) * 2,
                           uint64_t(c.es) * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
        else if (j.prod == kDown || j.prod == kDx)
            rc = encode_2d(&p.tmC[i], kF32, c.p, uint64_t(c.cols), uint64_t(c.rows), uint64_t(c.ld) * 4, 16, 32,
                           CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
        else
            rc = encode_2d(&p.tmC[i], f->dtype, c.p, uint64_t(c.cols), uint64_t(c.rows), uint64_t(c.ld) * 2, 32, 32,
                           CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
        p.out[i] = const_cast<void *>(c.p);
    }
    if (j.prod == kDh)
        for (int i = 0; i < 3 && rc == kOk; ++i)
            rc = encode_2d(&p.tmIn[i], f->dtype, j.in[i].p, uint64_t(j.in[i].cols), uint64_t(j.in[i].rows), uint64_t(j.in[i].ld) * 2, 32,
                           32, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    if (rc != kOk) return rc;
    const uint32_t b_bytes = b_mn ? uint32_t((b_rows + 63) / 64) * kPanel : uint32_t(b_rows) * 128u;
    p.stage_tx = 2u * (kSlot + b_bytes);
    // Instruction descriptor (layout as in tgemm.cu); bits 15 and 16 mark MN-major A and B.
    const uint32_t ab = f->dtype == kBF16 ? 1u : 0u;
    p.idesc = (1u << 4) | (ab << 7) | (ab << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
              (uint32_t(p.bn >> 3) << 17) | (uint32_t(256 >> 4) << 24);
    p.act = f->act;
    p.beside = j.beside;
    p.table = at.table;
    p.tiles = at.tiles;
    p.padded = at.padded;
    p.pair_of = at.pair_of;
    p.weights = j.weights;
    p.parts = j.parts;
    p.part_stride = j.part_stride;
    p.watchdog_ns = f->watchdog_ns;
    p.status = f->d_status;
    p.debug_stall = f->debug_stall;
    const unsigned grid = 2u * unsigned(most < f->pairs ? most : f->pairs);
    return launch(kExpertKernels[f->dtype == kBF16][j.prod], dim3(grid), dim3(kThreads), kExpertSmem[j.prod], s, 2, p);
}

// Dh's partial sums of dw: two warps share a tile's columns.
static int64_t dh_parts(int64_t hidden) { return 2 * ((hidden + 63) / 64); }

// The workspace, cut up: `end` is its size.
struct ExpertSpace {
    Placed at;
    char *xs, *dys, *h, *dg, *du, *hw;
    float *sums, *parts;
    int64_t end;
};

static ExpertSpace expert_space(char *base, const ExpertSizes &z, int64_t width, int64_t hidden, bool backward, bool own_h)
{
    ExpertSpace w{};
    auto take = [&](int64_t bytes) {
        char *p = base + w.end;
        w.end += (bytes + 255) / 256 * 256;
        return p;
    };
    auto ints = [&](int64_t n) { return reinterpret_cast<int *>(take(4 * n)); };
    const int64_t chunks = chunks_of(z);
    w.at.counts = ints(chunks > 1 ? (chunks + 1) * z.experts : 0);
    w.at.offsets = ints(z.experts + 1);
    w.at.padded = ints(z.experts + 1);
    w.at.tiles = ints(1);
    w.at.table = reinterpret_cast<RowTile *>(take(z.row_tiles * int64_t(sizeof(RowTile))));
    w.at.row_of = ints(z.pairs);
    w.at.pair_of = ints(z.padded_rows);
    w.xs = take(z.padded_rows * width * 2);
    w.sums = reinterpret_cast<float *>(take(z.padded_rows * width * 4));
    if (own_h) w.h = take(z.pairs * hidden * 2);
    if (backward) {
        w.dys = take(z.padded_rows * width * 2);
        w.dg = take(z.padded_rows * hidden * 2);
        w.du = take(z.padded_rows * hidden * 2);
        w.hw = take(z.padded_rows * hidden * 2);
        w.parts = reinterpret_cast<float *>(take(dh_parts(hidden) * z.padded_rows * 4));
    }
    return w;
}

static int check_stack(const Stack &a)
{
    if (!a.p || a.ld < a.cols || a.es < 0) return kErrInvalidArg;
    if (!aligned16(a.p) || a.ld % 8 || a.es % 8) return kErrAlignment;
    return kOk;
}

static int check_rows(const Mat &a)
{
    if (!a.p || a.ld < a.cols) return kErrInvalidArg;
    if (!aligned16(a.p) || a.ld % 8) return kErrAlignment;
    return kOk;
}

static int check_expert_sizes(int64_t tokens, int64_t experts, int top)
{
    if (tokens < 0 || experts < 1 || experts > kMostExperts || top < 1 || top > kMostTop) return kErrInvalidArg;
    // rows, rounded up to tiles, stay 32-bit
    if (tokens > 2147483647 / top || tokens * top + experts * kPadRows > 2147483647 - 2 * kRowTile) return kErrInvalidArg;
    return kOk;
}

static int zero(const Stack &c, int64_t experts, cudaStream_t s)
{
    if (c.p && cudaMemsetAsync(const_cast<void *>(c.p), 0, size_t(experts * c.rows * c.cols) * 2, s) != cudaSuccess) {
        cudaGetLastError();
        return kErrCuda;
    }
    return kOk;
}

}  // namespace tg

using namespace tg;

extern "C" {

int64_t tgemm_experts_workspace(tgemm_ffn_t f, int64_t tokens, int64_t experts, int top, int kind)
{
    if (!f || kind < TGEMM_EXPERTS_SERVE || kind > TGEMM_EXPERTS_BACKWARD) return -int64_t(kErrInvalidArg);
    const int rc = check_expert_sizes(tokens, experts, top);
    if (rc != kOk) return -int64_t(rc);
    return expert_space(nullptr, expert_sizes(tokens, experts, top), f->width, f->hidden, kind == TGEMM_EXPERTS_BACKWARD,
                        kind == TGEMM_EXPERTS_SERVE)
        .end;
}

int tgemm_experts_forward(tgemm_ffn_t f, int64_t tokens, int64_t experts, int top, const void *x, int64_t ldx, const int *chosen,
                          const float *weights, const void *w_gate, int64_t ld_gate, int64_t es_gate, const void *w_up,
                          int64_t ld_up, int64_t es_up, const void *w_down, int64_t ld_down, int64_t es_down, void *y,
                          int64_t ldy, void *g, void *u, void *h, void *workspace, int64_t workspace_bytes,
                          tgemm_stream_t stream)
{
    if (!f || !g != !u || !g != !h) return kErrInvalidArg;
    int rc = check_expert_sizes(tokens, experts, top);
    if (rc != kOk) return rc;
    if (tokens == 0) return kOk;
    const ExpertSizes z = expert_sizes(tokens, experts, top);
    const int64_t D = f->width, F = f->hidden, P = z.padded_rows;
    const Mat X{x, tokens, D, ldx}, Y{y, tokens, D, ldy};
    const Stack Wg{w_gate, F, D, ld_gate, es_gate}, Wu{w_up, F, D, ld_up, es_up}, Wd{w_down, D, F, ld_down, es_down};
    const ExpertSpace w = expert_space(static_cast<char *>(workspace), z, D, F, false, !h);
    const Stack H{h ? h : w.h, z.pairs, F, F, 0}, G{g ? g : H.p, z.pairs, F, F, 0}, U{u ? u : H.p, z.pairs, F, F, 0};
    if (!chosen || !weights || !workspace || workspace_bytes < w.end) return kErrInvalidArg;
    if (reinterpret_cast<uintptr_t>(chosen) % 4 || reinterpret_cast<uintptr_t>(weights) % 4 ||
        reinterpret_cast<uintptr_t>(workspace) % 256)
        return kErrAlignment;
    for (const Mat *m : {&X, &Y})
        if ((rc = check_rows(*m)) != kOk) return rc;
    for (const Stack *m : {&Wg, &Wu, &Wd, &H, &G, &U})
        if ((rc = check_stack(*m)) != kOk) return rc;
    if ((rc = experts_setup(f->dev)) != kOk) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Combine sum{w.sums, weights, y, ldy, nullptr, 0, 0, nullptr, nullptr, 0};
    if (!h && experts_are_few(z))
        return experts_few(ExpertsFewCall{x, ldx, D, F, chosen, {w_gate, w_up, w_down}, {ld_gate, ld_up, ld_down},
                                          {es_gate, es_up, es_down}, w.h, f->act},
                           sum, z, f->dev.sms, f->dtype == kBF16, s);
    if ((rc = experts_place(z, chosen, w.at, s)) != kOk) return rc;
    if ((rc = experts_gather(z, D, Gather{{x, nullptr}, {ldx, 0}, {w.xs, nullptr}}, w.at, s)) != kOk) return rc;
    ExpertJob up{kUp, 1, D, 1, 2, h ? 3 : 1, {{w.xs, P, D, D}}, {Wg, Wu}, {H, G, U}};
    if ((rc = expert_product(f, up, z, w.at, s)) != kOk) return rc;
    ExpertJob down{kDown, 1, F, 1, 1, 1, {{H.p, z.pairs, F, F}}, {Wd}, {{w.sums, P, D, D, 0}}};
    if ((rc = expert_product(f, down, z, w.at, s)) != kOk) return rc;
    return experts_combine(z, D, f->dtype == kBF16, sum, w.at, s);
}

int tgemm_experts_backward(tgemm_ffn_t f, int64_t tokens, int64_t experts, int top, const void *dy, int64_t lddy, const void *x,
                           int64_t ldx, const int *chosen, const float *weights, const void *w_gate, int64_t ld_gate,
                           int64_t es_gate, const void *w_up, int64_t ld_up, int64_t es_up, const void *w_down, int64_t ld_down,
                           int64_t es_down, const void *g, const void *u, const void *h, void *dx, int64_t lddx, float *dweights,
                           void *dw_gate, void *dw_up, void *dw_down, void *workspace, int64_t workspace_bytes,
                           tgemm_stream_t stream)
{
    if (!f) return kErrInvalidArg;
    int rc = check_expert_sizes(tokens, experts, top);
    if (rc != kOk) return rc;
    const int64_t D = f->width, F = f->hidden;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Stack dWg{dw_gate, F, D, D, F * D}, dWu{dw_up, F, D, D, F * D}, dWd{dw_down, D, F, F, D * F};
    const Stack *grads[] = {&dWg, &dWu, &dWd};
    for (const Stack *m : grads)
        if (m->p && (rc = check_stack(*m)) != kOk) return rc;
    if (tokens == 0) {  // empty sums
        for (const Stack *m : grads)
            if ((rc = zero(*m, experts, s)) != kOk) return rc;
        return kOk;
    }
    const ExpertSizes z = expert_sizes(tokens, experts, top);
    const int64_t P = z.padded_rows;
    const Mat X{x, tokens, D, ldx}, dY{dy, tokens, D, lddy}, dX{dx, tokens, D, lddx};
    const Mat H{h, z.pairs, F, F}, G{g, z.pairs, F, F}, U{u, z.pairs, F, F};
    const Stack Wg{w_gate, F, D, ld_gate, es_gate}, Wu{w_up, F, D, ld_up, es_up}, Wd{w_down, D, F, ld_down, es_down};
    const ExpertSpace w = expert_space(static_cast<char *>(workspace), z, D, F, true, false);
    if (!chosen || !weights || !workspace || workspace_bytes < w.end) return kErrInvalidArg;
    if (reinterpret_cast<uintptr_t>(chosen) % 4 || reinterpret_cast<uintptr_t>(weights) % 4 ||
        reinterpret_cast<uintptr_t>(dweights) % 4 || reinterpret_cast<uintptr_t>(workspace) % 256)
        return kErrAlignment;
    for (const Mat *m : {&X, &dY, &H, &G, &U})
        if ((rc = check_rows(*m)) != kOk) return rc;
    if (dx && (rc = check_rows(dX)) != kOk) return rc;
    for (const Stack *m : {&Wg, &Wu, &Wd})
        if ((rc = check_stack(*m)) != kOk) return rc;
    if ((rc = experts_setup(f->dev)) != kOk) return rc;
    if ((rc = experts_place(z, chosen, w.at, s)) != kOk) return rc;
    if ((rc = experts_gather(z, D, Gather{{dy, x}, {lddy, ldx}, {w.dys, w.xs}}, w.at, s)) != kOk) return rc;
    ExpertJob dh{kDh, 1, D, 1, 1, 3, {{w.dys, P, D, D}}, {Wd}, {{w.dg, P, F, F, 0}, {w.du, P, F, F, 0}, {w.hw, P, F, F, 0}}};
    dh.in[0] = G;
    dh.in[1] = U;
    dh.in[2] = H;
    dh.weights = weights;
    dh.parts = w.parts;
    dh.part_stride = P;
    if ((rc = expert_product(f, dh, z, w.at, s)) != kOk) return rc;
    if (dx) {
        ExpertJob j{kDx, 1, F, 2, 2, 1, {{w.dg, P, F, F}, {w.du, P, F, F}}, {Wg, Wu}, {{w.sums, P, D, D, 0}}};
        j.shared = dw_gate || dw_up || dw_down;
        if ((rc = expert_product(f, j, z, w.at, s)) != kOk) return rc;
    }
    ExpertJob dw{kDw, 0, 0, 0, 0, 0, {}, {}, {}};
    const Mat as[] = {{w.dg, P, F, F}, {w.du, P, F, F}, {w.dys, P, D, D}};
    const Stack bs[] = {{w.xs, P, D, D, 0}, {w.xs, P, D, D, 0}, {w.hw, P, F, F, 0}};
    for (int i = 0; i < 3; ++i) {
        if (!grads[i]->p) continue;
        dw.A[dw.problems] = as[i];
        dw.B[dw.problems] = bs[i];
        dw.C[dw.problems++] = *grads[i];
    }
    dw.na = dw.nb = dw.nc = dw.problems;
    dw.beside = dw.shared = dx != nullptr;
    if (dw.problems && (rc = expert_product(f, dw, z, w.at, s)) != kOk) return rc;
    if (!dx && !dweights) return kOk;
    const int width = expert_tile_width(f, dh, z, int((D + kBlockK - 1) / kBlockK));
    const Combine c{w.sums, nullptr, dx, lddx, w.parts, P, int(2 * ((F + width - 1) / width)), dweights, nullptr, 0};
    return experts_combine(z, D, f->dtype == kBF16, c, w.at, s);
}

}  // extern "C"
