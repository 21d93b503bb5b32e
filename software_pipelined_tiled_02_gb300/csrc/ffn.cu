// ffn.cu -- a transformer's gated feed-forward block, forward and backward,
// for GB300 (sm_103a), and its C ABI.
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u,  y = h Wd^T
//   dh = dy Wd,  dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h
// with x, y: [tokens, width], Wg, Wu: [hidden, width], Wd: [width, hidden],
// all row-major, fp16 or bf16, every sum in fp32.
//
// Five products on the tensor cores, each one launch of ffn_gemm_kernel:
//   Up    g, u and h together.  A CTA pair's 256 columns are 128 (or fewer)
//         of Wg in the even CTA and the same ones of Wu in the odd: one MMA
//         computes both projections, and a thread of the epilogue finds g and
//         u of its element in two columns of its tensor-memory lane.
//   Down  y.
//   Dh    dh, whose epilogue reads g and u and writes dg and du; dh itself is
//         never rounded or stored.
//   Dx    dx, one K loop over dg Wg and then du Wu into one accumulator.
//   Dw    dWg, dWu and dWd as one list of tiles.
// Wd in Dh, Wg and Wu in Dx, and all operands of Dw have the reduction index
// as their row index ("MN-major"): they are loaded as they lie, as boxes of 64
// columns x 64 reduction rows, and the tensor core reads them transposed.
//
// The pipeline is tgemm.cu's: a ring of slots of 64 reduction elements, filled by
// TMA (warp 0: A, warp 10: B), read by tcgen05.mma (warp 1) on CTA pairs with 256
// rows a tile, drained by warps 2 .. 9 from one of two tensor-memory accumulators
// while the next tile's MMAs fill the other.
//
// What bounds it, at 4096 tokens, 2048 x 8192 bf16 (tensor pipe active, share of
// cycles): Up 153 us (90 %), Down 81 us (90 %), Dx 157 us (95 %), Dw 226 us (93 %);
// Dh 94 us (70 %), whose epilogue moves four tensors of C's size for a K of the
// width alone.  8192 tokens, 4096 x 8192, call after call under the power cap: 970
// to 995 us forward, 2.04 to 2.09 ms backward, 1.6 to 1.7 PFLOP/s; the first passes
// after a pause, at full clocks: 858 us and 1.82 ms.  With few tiles a K block
// costs 235 ns at any width up to 192 columns: a producer's load and the MMA warp's
// wait, MMAs and commit take about that long each.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>
#include <new>

#include "ffn.cuh"
#include "host.h"
#include "layout.h"
#include "ptx.cuh"
#include "tgemm.h"
#include "watchdog.cuh"

namespace tg {

constexpr uint32_t kStageBuf = 32 * 64;     // a box of an epilogue warp: 32 rows of 64 bytes (32 columns)

// A product's shared memory: the ring's A slots, its B slots, the epilogue
// warps' boxes (two going out; Dh also two coming in, of g and u, and one slot
// less for them), the barriers.
template <int PROD>
struct FfnLayout {
    static constexpr int kStages = PROD == kDh ? 5 : 6;
    static constexpr int kBoxes = PROD == kDh ? 4 : 2;  // per epilogue warp
    static constexpr uint32_t kOffB = kStages * kSlot, kOffC = 2 * kStages * kSlot;
    static constexpr uint32_t kOffBar = kOffC + kBoxes * kEpiWarps * kStageBuf;
    static constexpr int kBars = 2 * kStages + 6 + kEpiWarps;
    static constexpr uint32_t kTotal = kOffBar + 8 * kBars + 16 + kSmemAlign;
};
constexpr uint32_t kFfnSmem = FfnLayout<kUp>::kTotal > FfnLayout<kDh>::kTotal ? FfnLayout<kUp>::kTotal : FfnLayout<kDh>::kTotal;
constexpr int kAccCols = 256;               // tensor-memory columns between the two accumulators

struct FfnParams {  // 64-byte aligned through its CUtensorMap members
    // Operands and outputs by index: Up reads B by CTA rank (gate, up) and
    // stores h, g, u; Dh stores dg, du; Dx reads A and B by K segment; Dw
    // reads and stores by problem.
    CUtensorMap tmA[3], tmB[3], tmC[3];
    int m[3], n[3];               // rows and columns of each problem's output
    int tiles_m[3], tiles_n[3];
    int first_tile[4];            // first tile index of each problem, then the total
    int problems;
    int bn;                       // columns of a tile: Up counts both projections
    int tile_cols;                // output columns of a tile: bn, or bn / 2 for Up
    int num_kb;                   // 64-element reduction blocks per tile
    int seg_kb;                   // Dx: blocks of its first K segment
    int group_m;
    uint32_t idesc;
    uint32_t stage_tx;            // bytes both CTAs' loads deliver per slot
    int act, save;
    int beside;                   // Dw: see Job
    CUtensorMap tmG, tmU;         // Dh: the projections
    unsigned long long watchdog_ns;
    int *status;
    int debug_stall;
};

// ---------------------------------------------------------------- the tiled products

struct Tile {
    int prob, mb, nb;
};

// Tile t of the list: its problem, then grouped raster order inside it.
__device__ __forceinline__ Tile tile_at(const FfnParams &p, int t)
{
    Tile w;
    w.prob = 0;
    while (w.prob + 1 < p.problems && t >= p.first_tile[w.prob + 1]) ++w.prob;
    const int r0 = t - p.first_tile[w.prob];
    const int per_group = p.group_m * p.tiles_n[w.prob];
    const int grp = r0 / per_group, first_m = grp * p.group_m;
    const int gm = min(p.group_m, p.tiles_m[w.prob] - first_m);
    const int r = r0 - grp * per_group;
    w.mb = first_m + r % gm;
    w.nb = r / gm;
    return w;
}

template <int PROD, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) ffn_gemm_kernel(const __grid_constant__ FfnParams p)
{
    constexpr bool A_MN = PROD == kDw, B_MN = PROD == kDh || PROD == kDx || PROD == kDw;
    using L = FfnLayout<PROD>;
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
    auto box_in = [&](int w) { return bars + 8u * uint32_t(2 * kStages + 6 + w); };  // Dh: epilogue warp w's g and u
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffBar + 8 * L::kBars);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32;
    const uint32_t rank = cluster_ctarank();
    const int pair = int(blockIdx.x >> 1), pairs = int(gridDim.x >> 1);
    const int tiles = p.first_tile[p.problems];

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

    if (warp == 0 || warp == kProducerBWarp) {
        // Producers: one lane each, up to kStages slots ahead (tgemm.cu).  Each
        // CTA loads its 128 rows of A and its half of B's columns; both complete
        // the even CTA's full[s].
        if (lane == 0) {
            const uint32_t full_leader = map_to_rank(full(0), 0);
            const int b_rows = p.bn / 2;
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {  // a wait that fails ends the loop
                const Tile w = tile_at(p, t);
                const int m0 = w.mb * 256 + int(rank) * 128;
                const int n0 = PROD == kUp ? w.nb * p.tile_cols : w.nb * p.bn + int(rank) * b_rows;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_try_wait(empty(s), ph ^ 1u) && !wait_bar(empty(s), ph ^ 1u, p, abort, 0, issued)) {
                        ok = false;
                        break;
                    }
                    const int seg = PROD == kDx && kb >= p.seg_kb ? 1 : 0;
                    const int k = (kb - (seg ? p.seg_kb : 0)) * kBlockK;
                    const int ia = PROD == kDw ? w.prob : seg;
                    const int ib = PROD == kUp ? int(rank) : ia;
                    if (!check(s < kStages && w.mb < p.tiles_m[w.prob] && w.nb < p.tiles_n[w.prob] && n0 % 8 == 0, p,
                               abort, 0, issued)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full_leader + 8u * uint32_t(s);
                    if (warp == 0) {
                        const uint32_t dst = sA + uint32_t(s) * kSlot;
                        if (rank == 0) mbar_arrive_expect_tx(full(s), p.stage_tx);
                        if constexpr (A_MN) {
                            tma_load_2d_pair(dst, &p.tmA[ia], m0, k, bar);
                            tma_load_2d_pair(dst + kPanel, &p.tmA[ia], m0 + 64, k, bar);
                        } else {
                            tma_load_2d_pair(dst, &p.tmA[ia], k, m0, bar);
                        }
                    } else {
                        const uint32_t dst = sB + uint32_t(s) * kSlot;
                        if constexpr (B_MN) {
                            tma_load_2d_pair(dst, &p.tmB[ib], n0, k, bar);
                            if (b_rows > 64) tma_load_2d_pair(dst + kPanel, &p.tmB[ib], n0 + 64, k, bar);
                        } else {
                            tma_load_2d_pair(dst, &p.tmB[ib], k, n0, bar);
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
            // 16 reduction elements further on, in 16-byte units: 32 bytes along a
            // K-major swizzle row, or two groups of 8 swizzle rows
            constexpr uint64_t a_step = A_MN ? 2048 >> 4 : 32 >> 4, b_step = B_MN ? 2048 >> 4 : 32 >> 4;
            int s = 0, a = 0, it = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            if (p.debug_stall) ok = warp_wait(stall, 0, p, abort, 1, 0);  // test hook: nothing arrives
            for (int t = pair; ok && t < tiles; t += pairs) {
                if (!warp_wait(acc_empty(a), aph ^ 1u, p, abort, 1, it)) break;
                tc_fence_after();
                const uint32_t d = tmem + uint32_t(a * kAccCols);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!warp_wait(full(s), ph, p, abort, 1, it)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = ad0 + uint64_t(s) * (kSlot >> 4), bd = bd0 + uint64_t(s) * (kSlot >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBlockK / 16; ++kk)
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
        const uint32_t my_bufs = sC + uint32_t(L::kBoxes * (warp - 2)) * kStageBuf;
        uint32_t boxes = 0, aph = 0;
        int a = 0, done = 0;
        // Stage 32 columns of this lane's row (16 packed words) in buffer k, and
        // store the boxes staged so: their buffers are free once earlier stores have
        // read them.
        auto stage = [&](int k, const uint32_t (&w)[16]) {
            const uint32_t at = my_bufs + uint32_t(k) * kStageBuf + uint32_t(lane) * 64u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                st_shared_v4(at + (uint32_t(j ^ ((lane >> 1) & 3)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2],
                             w[4 * j + 3]);
        };
        [[maybe_unused]] auto put = [&](const CUtensorMap *map, int col, int row, const uint32_t (&w)[16]) {
            const int k = int(boxes & 1u);
            if (boxes >= 2u && lane == 0) bulk_wait_read<PROD == kUp ? 0 : 1>();
            __syncwarp();
            stage(k, w);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, col, row, my_bufs + uint32_t(k) * kStageBuf);
                bulk_commit();
            }
            ++boxes;
        };
        // Two boxes of the same place in two outputs, with one fence.
        [[maybe_unused]] auto put_both = [&](const CUtensorMap *map0, const CUtensorMap *map1, int col, int row, const uint32_t (&w0)[16],
                            const uint32_t (&w1)[16]) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            stage(0, w0);
            stage(1, w1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map0, col, row, my_bufs);
                tma_store_2d(map1, col, row, my_bufs + kStageBuf);
                bulk_commit();
            }
            boxes = 2;  // put() goes on with buffer 0 and waits for these stores
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
        auto row_of = [&](const Tile &w) { return w.mb * 256 + int(rank) * 128 + q * 32; };
        // Dh: this warp's boxes of g and u for its next chunk, on their way while
        // the current one is worked on (or its tile's sums are still forming).
        [[maybe_unused]] const uint32_t in_bar = box_in(warp - 2), in_g = my_bufs + 2 * kStageBuf, in_u = in_g + kStageBuf;
        [[maybe_unused]] uint32_t in_ph = 0;
        [[maybe_unused]] bool coming = false;
        [[maybe_unused]] auto fetch = [&](const Tile &w, int c) -> bool {
            const int col = w.nb * p.tile_cols + c * 32;
            if (c * 32 >= p.tile_cols || row_of(w) >= p.m[0] || col >= p.n[0]) return false;
            __syncwarp();  // every lane has read the boxes
            if (lane == 0) {
                mbar_arrive_expect_tx(in_bar, 2 * kStageBuf);
                tma_load_2d(in_g, &p.tmG, col, row_of(w), in_bar);
                tma_load_2d(in_u, &p.tmU, col, row_of(w), in_bar);
            }
            coming = true;
            return true;
        };
        if constexpr (PROD == kDh) {
            if (pair < tiles) fetch(tile_at(p, pair), sub);
        }
        for (int t = pair; t < tiles; t += pairs, ++done) {
            const Tile w = tile_at(p, t);
            const int row0 = row_of(w), n0 = w.nb * p.tile_cols;
            const int m = p.m[w.prob], n = p.n[w.prob];
            if (!warp_wait(acc_full(a), aph, p, abort, 2, done)) break;
            tc_fence_after();
            const uint32_t acc = uint32_t(a * kAccCols);
            for (int c = sub; c * 32 < p.tile_cols && row0 < m && n0 + c * 32 < n; c += 2) {
                const int col = n0 + c * 32;
                if (!check(int(acc) + (PROD == kUp ? p.tile_cols : 0) + (c + 1) * 32 <= kTmemColsMax && col % 8 == 0, p,
                           abort, 2, done))
                    break;
                uint32_t o[16];
                if constexpr (PROD == kUp) {
                    float g[32], u[32];
                    read(acc + uint32_t(c * 32), g);
                    read(acc + uint32_t(p.tile_cols + c * 32), u);
                    if (p.save) {
                        uint32_t o_u[16];
                        packed(g, o);
                        packed(u, o_u);
                        put_both(&p.tmC[1], &p.tmC[2], col, row0, o, o_u);
                    }
                    auto gate = [&](auto act_c) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            F2 act, slope;
                            activate<decltype(act_c)::value>(f2(g[e], g[e + 1]), act, slope);
                            o[e / 2] = pack2(act * f2(u[e], u[e + 1]), BF16);
                        }
                    };
                    if (p.act == kSilu)
                        gate(std::integral_constant<int, kSilu>{});
                    else if (p.act == kGelu)
                        gate(std::integral_constant<int, kGelu>{});
                    else
                        gate(std::integral_constant<int, kRelu>{});
                    put(&p.tmC[0], col, row0, o);
                } else if constexpr (PROD == kDh) {
                    // g and u of this lane's row; then the boxes take the next chunk's
                    if (!warp_wait(in_bar, in_ph, p, abort, 2, done)) break;
                    in_ph ^= 1u;
                    coming = false;
                    uint4 gq[4], uq[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t at = uint32_t(lane) * 64u + (uint32_t(j ^ ((lane >> 1) & 3)) << 4);
                        gq[j] = ld_shared_v4(in_g + at);
                        uq[j] = ld_shared_v4(in_u + at);
                    }
                    if (!fetch(w, c + 2) && t + pairs < tiles) fetch(tile_at(p, t + pairs), sub);
                    float dh[32];
                    read(acc + uint32_t(c * 32), dh);
                    uint32_t dg[16];
                    auto ungate = [&](auto act_c) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint32_t gw = (&gq[j / 4].x)[j % 4], uw = (&uq[j / 4].x)[j % 4];
                            const float2 g2 = unpack2(gw, BF16), u2 = unpack2(uw, BF16);
                            const F2 d = f2(dh[2 * j], dh[2 * j + 1]);
                            F2 act, slope;
                            activate<decltype(act_c)::value>(f2(g2.x, g2.y), act, slope);
                            dg[j] = pack2(d * f2(u2.x, u2.y) * slope, BF16);
                            o[j] = pack2(d * act, BF16);
                        }
                    };
                    if (p.act == kSilu)
                        ungate(std::integral_constant<int, kSilu>{});
                    else if (p.act == kGelu)
                        ungate(std::integral_constant<int, kGelu>{});
                    else
                        ungate(std::integral_constant<int, kRelu>{});
                    put_both(&p.tmC[0], &p.tmC[1], col, row0, dg, o);
                } else {
                    float v[32];
                    read(acc + uint32_t(c * 32), v);
                    packed(v, o);
                    put(&p.tmC[PROD == kDw ? w.prob : 0], col, row0, o);
                }
            }
            if constexpr (PROD == kDh) {  // no chunk of this tile was this warp's: the next tile's boxes were not asked for
                if (!coming && t + pairs < tiles) fetch(tile_at(p, t + pairs), sub);
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

}  // namespace tg

// ---------------------------------------------------------------- host side

using namespace tg;

namespace tg {

typedef void (*FfnKernel)(const FfnParams);
static const FfnKernel kFfnKernels[2][5] = {  // by type (fp16, bf16) and product
    {ffn_gemm_kernel<kUp, false>, ffn_gemm_kernel<kDown, false>, ffn_gemm_kernel<kDh, false>, ffn_gemm_kernel<kDx, false>,
     ffn_gemm_kernel<kDw, false>},
    {ffn_gemm_kernel<kUp, true>, ffn_gemm_kernel<kDown, true>, ffn_gemm_kernel<kDh, true>, ffn_gemm_kernel<kDx, true>,
     ffn_gemm_kernel<kDw, true>}};

// Once per device: the kernels' shared-memory ceiling, and how many CTA pairs
// are resident at once.
static int ffn_setup(const Device &d, int *pairs)
{
    static std::mutex mu;
    static int known[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (d.ordinal < 64 && known[d.ordinal]) {
        *pairs = known[d.ordinal];
        return kOk;
    }
    if (int(kFfnSmem) > d.smem_limit) return kErrSmemBudget;
    for (const auto &type : kFfnKernels) {
        for (FfnKernel k : type) {
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kFfnSmem)) != cudaSuccess) {
                cudaGetLastError();
                return kErrCuda;
            }
        }
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(2 * (d.sms / 2)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kFfnSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kFfnKernels[0][0], &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return kErrCuda;
    }
    if (d.ordinal < 64) known[d.ordinal] = n;
    *pairs = n;
    return kOk;
}

// An operand whose tile is `tile_rows` output rows (or columns) in this CTA.
// K-major: the reduction runs along the matrix's rows; MN-major: down them.
static int operand_map(CUtensorMap *m, int dtype, const Mat &a, bool mn, int tile_rows)
{
    const uint64_t pitch = uint64_t(a.ld) * 2;
    return encode_2d(m, dtype, a.p, uint64_t(a.cols), uint64_t(a.rows), pitch, 64, mn ? 64u : uint32_t(tile_rows),
                     CU_TENSOR_MAP_SWIZZLE_128B, operand_promotion(pitch));
}

// Boxes of 32 rows and 32 columns, as an epilogue warp stores (or loads) them.
static int output_map(CUtensorMap *m, int dtype, const Mat &c)
{
    return encode_2d(m, dtype, c.p, uint64_t(c.cols), uint64_t(c.rows), uint64_t(c.ld) * 2, 32, 32,
                     CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// Columns of a tile: the width with the least estimated time in SM cycles, whole
// waves of tiles times a tile's.  A 64-element block takes about 580 at any width:
// 512 are the MMAs of 256 columns, and fewer columns cost little less (see the top
// of this file).  A tile's hand-over and epilogue take 2000
// and 18 a column, set-up 6000.  Dx and Dw run beside each other: a block then
// takes 260 and 1.7 a column, and 630 at least, and a product's share of the
// machine counts too (1001 tokens, 520 x 1400, run their backward pass in 30 us
// with Dx in 192 columns and Dw in 256, and in 35 to 42 us with the cuts that are
// quickest for either alone).
//   The constants here and in ffn_few.cu are those whose choice came nearest to
// the fastest of up to 200 combinations of cuts of whole passes (52 sizes of 1 to
// 8192 tokens, 128 x 128 to 4096 x 8192): 1.5 % slower on average forward and
// 3.2 % backward, 9 % and 17 % at most.
static int tile_width(const tgemm_ffn_s *f, const Job &j, int num_kb, double *cycles)
{
    int best = 256;
    double best_cost = 0.0;
    for (int bn = 256; bn >= 64; bn -= 32) {
        if (j.prod == kUp && bn % 64) continue;  // whole 32-column chunks of both projections
        const int cols = j.prod == kUp ? bn / 2 : bn;
        int64_t tiles = 0;
        for (int i = 0; i < j.problems; ++i)
            tiles += (j.C[i].rows + 255) / 256 * ((j.C[i].cols + cols - 1) / cols);
        const int64_t waves = (tiles + f->pairs - 1) / f->pairs;
        const double beside = 260.0 + 1.7 * bn > 630.0 ? 260.0 + 1.7 * bn : 630.0;
        const double tile = (j.shared ? beside : 580.0) * num_kb + 2000.0 + 18.0 * bn;
        double cost = double(waves) * tile + 6000.0;
        if (j.shared) cost += kShare * double(tiles) * tile / f->pairs;
        if (bn == 256 || cost < best_cost) {
            best = bn;
            best_cost = cost;
        }
    }
    *cycles = best_cost;
    return best;
}

// How a product is cut up: by the kernels of ffn_few.cu where they are estimated
// quicker.  At 4096 x 8192 bf16 they win for Up, Down, Dh and Dx up to 128 tokens
// (64 tokens: forward 42.8 us against 58.6 here), for some of those up to 256, and
// beyond that where this file's kernel has tiles for a part of the SMs only (8000
// tokens, 128 x 128: backward 17 us against 45); with tiles for all SMs this kernel
// wins (384 tokens, 8192 x 8192: forward 118 us against 167).
struct Cut {
    bool few;
    FewShape shape;       // few
    int bn, seg_kb, num_kb;  // otherwise
};

static Cut ffn_cut(const tgemm_ffn_s *f, const Job &j)
{
    Cut c{};
    c.seg_kb = int((j.k + kBlockK - 1) / kBlockK);
    c.num_kb = j.prod == kDx ? 2 * c.seg_kb : c.seg_kb;
    double cycles = 0.0, few_cycles = 0.0;
    c.bn = tile_width(f, j, c.num_kb, &cycles);
    c.shape = ffn_few_shape(f, j, &few_cycles);
    c.few = few_cycles < cycles;
    return c;
}

// One to eight tokens and few weights: launch latency counts, and the kernels
// without tensor memory, barriers or tensor maps are quicker (one token: 512 x
// 2048 6.2 us against 8.9 us; 1024 x 4096 12.4 against 12.0; 4096 x 8192 43.4
// against 39.7).
static bool ffn_takes_rows(const tgemm_ffn_s *f, int64_t tokens)
{
    return tokens <= kRowsTokens && f->width * f->hidden <= int64_t(1) << 21;
}

static int ffn_product(tgemm_ffn_s *f, const Job &j, cudaStream_t s)
{
    const Cut cut = ffn_cut(f, j);
    if (cut.few) return ffn_few_product(f, j, cut.shape, s);
    FfnParams p;
    std::memset(&p, 0, sizeof(p));
    p.save = j.nc == 3 && j.prod == kUp;
    const bool a_mn = j.prod == kDw, b_mn = j.prod == kDh || j.prod == kDx || j.prod == kDw;
    p.problems = j.problems;
    p.seg_kb = cut.seg_kb;
    p.num_kb = cut.num_kb;
    p.bn = cut.bn;
    p.tile_cols = j.prod == kUp ? p.bn / 2 : p.bn;
    p.group_m = 8;
    int64_t total = 0;
    for (int i = 0; i < j.problems; ++i) {
        p.m[i] = int(j.C[i].rows);
        p.n[i] = int(j.C[i].cols);
        const int64_t tm = (j.C[i].rows + 255) / 256, tn = (j.C[i].cols + p.tile_cols - 1) / p.tile_cols;
        p.tiles_m[i] = int(tm);
        p.tiles_n[i] = int(tn);
        p.first_tile[i] = int(total);
        total += tm * tn;
    }
    if (total > (int64_t(1) << 30)) return kErrInvalidArg;
    p.first_tile[j.problems] = int(total);
    const int b_rows = p.bn / 2;
    int rc = kOk;
    for (int i = 0; i < j.na && rc == kOk; ++i) rc = operand_map(&p.tmA[i], f->dtype, j.A[i], a_mn, 128);
    for (int i = 0; i < j.nb && rc == kOk; ++i) rc = operand_map(&p.tmB[i], f->dtype, j.B[i], b_mn, b_rows);
    for (int i = 0; i < j.nc && rc == kOk; ++i) rc = output_map(&p.tmC[i], f->dtype, j.C[i]);
    if (rc != kOk) return rc;
    const uint32_t b_bytes = b_mn ? uint32_t((b_rows + 63) / 64) * kPanel : uint32_t(b_rows) * 128u;
    p.stage_tx = 2u * (kSlot + b_bytes);
    // Instruction descriptor (layout as in tgemm.cu); bits 15 and 16 mark MN-major A and B.
    const uint32_t ab = f->dtype == kBF16 ? 1u : 0u;
    p.idesc = (1u << 4) | (ab << 7) | (ab << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
              (uint32_t(p.bn >> 3) << 17) | (uint32_t(256 >> 4) << 24);
    if (j.prod == kDh) {
        for (int i = 0; i < 2 && rc == kOk; ++i) {
            Mat a = j.C[0];
            a.p = i ? j.u : j.g;
            rc = output_map(i ? &p.tmU : &p.tmG, f->dtype, a);
        }
        if (rc != kOk) return rc;
    }
    p.act = f->act;
    p.beside = j.beside;
    p.watchdog_ns = f->watchdog_ns;
    p.status = f->d_status;
    p.debug_stall = f->debug_stall;
    const unsigned grid = 2u * unsigned(total < f->pairs ? total : f->pairs);
    return launch(kFfnKernels[f->dtype == kBF16][j.prod], dim3(grid), dim3(kThreads), kFfnSmem, s, 2, p);
}

// While it lives, this thread may allocate and free device memory although a
// stream is being captured: what a plan owns is no part of the captured work.
struct OutsideCapture {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
    ~OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// A plan's status word, zero before this returns: it is cleared on a stream of
// its own, because a plan's first launch may go to a stream that does not wait
// for the default one.
static int status_word(int **out)
{
    const OutsideCapture relaxed;
    int *p = nullptr;
    cudaStream_t s = nullptr;
    bool ok = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) == cudaSuccess &&
              cudaMalloc(&p, 4 * sizeof(int)) == cudaSuccess && cudaMemsetAsync(p, 0, 4 * sizeof(int), s) == cudaSuccess &&
              cudaStreamSynchronize(s) == cudaSuccess;
    if (s && cudaStreamDestroy(s) != cudaSuccess) ok = false;
    if (!ok) {
        cudaGetLastError();
        if (p) cudaFree(p);
        return kErrCuda;
    }
    *out = p;
    return kOk;
}

// What every matrix argument has to meet: given, 16-byte aligned, rows that do
// not overlap and start on 16-byte boundaries.
static int check_mat(const Mat &a)
{
    if (!a.p || a.ld < a.cols) return kErrInvalidArg;
    if (!aligned16(a.p) || a.ld % 8) return kErrAlignment;
    return kOk;
}

static int check_mats(const Mat *const *list, int n)
{
    for (int i = 0; i < n; ++i) {
        const int rc = check_mat(*list[i]);
        if (rc != kOk) return rc;
    }
    return kOk;
}

}  // namespace tg

constexpr int64_t kMaxTokens = 2147483647 - 257;  // a coordinate rounded up to a tile stays 32-bit
constexpr int64_t kMaxFeatures = int64_t(1) << 24;

extern "C" {

int tgemm_ffn_validate(int64_t width, int64_t hidden, int dtype, int activation)
{
    if (dtype != kF16 && dtype != kBF16) return kErrUnsupportedDtype;
    if (width < 1 || hidden < 1 || width > kMaxFeatures || hidden > kMaxFeatures) return kErrInvalidArg;
    if (activation != kSilu && activation != kGelu && activation != kRelu) return kErrInvalidArg;
    if (width % 8 || hidden % 8) return kErrAlignment;
    return kOk;
}

int tgemm_ffn_plan(tgemm_ffn_t *out, int64_t width, int64_t hidden, int dtype, int activation)
{
    if (!out) return kErrInvalidArg;
    *out = nullptr;
    int rc = tgemm_ffn_validate(width, hidden, dtype, activation);
    if (rc != kOk) return rc;
    Device d;
    if ((rc = current_device(d)) != kOk) return rc;
    if (!d.gb300) return kErrArch;
    int pairs = 0;
    if ((rc = ffn_setup(d, &pairs)) != kOk) return rc;
    tgemm_ffn_s *f = new (std::nothrow) tgemm_ffn_s();
    if (!f) return kErrCuda;
    f->width = width;
    f->hidden = hidden;
    f->dtype = dtype;
    f->act = activation;
    f->dev = d;
    f->pairs = pairs;
    f->watchdog_ns = env_watchdog();
    f->debug_stall = 0;
    if (status_word(&f->d_status) != kOk) {
        delete f;
        return kErrCuda;
    }
    *out = f;
    return kOk;
}

int tgemm_ffn_forward(tgemm_ffn_t f, int64_t tokens, const void *x, int64_t ldx, const void *w_gate, int64_t ld_gate,
                      const void *w_up, int64_t ld_up, const void *w_down, int64_t ld_down, void *y, int64_t ldy,
                      void *g, void *u, void *h, tgemm_stream_t stream)
{
    if (!f || tokens < 0 || tokens > kMaxTokens || !g != !u) return kErrInvalidArg;
    if (tokens == 0) return kOk;
    const int64_t D = f->width, F = f->hidden;
    const Mat X{x, tokens, D, ldx}, Wg{w_gate, F, D, ld_gate}, Wu{w_up, F, D, ld_up}, Wd{w_down, D, F, ld_down};
    const Mat Y{y, tokens, D, ldy}, H{h, tokens, F, F}, G{g ? g : h, tokens, F, F}, U{u ? u : h, tokens, F, F};
    const Mat *all[] = {&X, &Wg, &Wu, &Wd, &Y, &H, &G, &U};
    int rc = check_mats(all, 8);
    if (rc != kOk) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (ffn_takes_rows(f, tokens))
        return ffn_rows_forward(FfnRows{int(tokens), D, F, ldx, ld_gate, ld_up, ld_down, ldy, x, w_gate, w_up, w_down, y, g,
                                        u, h, f->dtype == kBF16, f->act},
                                s);
    Job up{kUp, 1, D, 1, 2, g ? 3 : 1, {X}, {Wg, Wu}, {H, G, U}};
    if ((rc = ffn_product(f, up, s)) != kOk) return rc;
    Job down{kDown, 1, F, 1, 1, 1, {H}, {Wd}, {Y}};
    return ffn_product(f, down, s);
}

int tgemm_ffn_backward(tgemm_ffn_t f, int64_t tokens, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                       const void *w_gate, int64_t ld_gate, const void *w_up, int64_t ld_up, const void *w_down,
                       int64_t ld_down, const void *g, const void *u, const void *h, void *dx, int64_t lddx,
                       void *dw_gate, void *dw_up, void *dw_down, void *dg, void *du, tgemm_stream_t stream)
{
    if (!f || tokens < 0 || tokens > kMaxTokens) return kErrInvalidArg;
    const int64_t D = f->width, F = f->hidden;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int rc = kOk;
    const Mat dWg{dw_gate, F, D, D}, dWu{dw_up, F, D, D}, dWd{dw_down, D, F, F};
    const Mat *grads[] = {&dWg, &dWu, &dWd};
    for (const Mat *m : grads)
        if (m->p && (rc = check_mat(*m)) != kOk) return rc;
    if (tokens == 0) {  // empty sums
        for (const Mat *m : grads) {
            if (m->p && cudaMemsetAsync(const_cast<void *>(m->p), 0, size_t(F) * size_t(D) * 2, s) != cudaSuccess) {
                cudaGetLastError();
                return kErrCuda;
            }
        }
        return kOk;
    }
    const Mat X{x, tokens, D, ldx}, Wg{w_gate, F, D, ld_gate}, Wu{w_up, F, D, ld_up}, Wd{w_down, D, F, ld_down};
    const Mat dY{dy, tokens, D, lddy}, G{g, tokens, F, F}, U{u, tokens, F, F}, H{h, tokens, F, F};
    const Mat dG{dg, tokens, F, F}, dU{du, tokens, F, F}, dX{dx, tokens, D, lddx};
    const Mat *all[] = {&X, &Wg, &Wu, &Wd, &dY, &G, &U, &H, &dG, &dU};
    if ((rc = check_mats(all, 10)) != kOk) return rc;
    if (dx && (rc = check_mat(dX)) != kOk) return rc;
    Job dh{kDh, 1, D, 1, 1, 2, {dY}, {Wd}, {dG, dU}, g, u};
    if ((rc = ffn_product(f, dh, s)) != kOk) return rc;
    const bool shared = dx && (grads[0]->p || grads[1]->p || grads[2]->p);
    if (dx) {
        Job j{kDx, 1, F, 2, 2, 1, {dG, dU}, {Wg, Wu}, {dX}};
        j.shared = shared;
        if ((rc = ffn_product(f, j, s)) != kOk) return rc;
    }
    Job dw{kDw, 0, tokens, 0, 0, 0, {}, {}, {}};
    const Mat as[] = {dG, dU, dY}, bs[] = {X, X, H};
    for (int i = 0; i < 3; ++i) {
        if (!grads[i]->p) continue;
        dw.A[dw.problems] = as[i];
        dw.B[dw.problems] = bs[i];
        dw.C[dw.problems++] = *grads[i];
    }
    dw.na = dw.nb = dw.nc = dw.problems;
    dw.beside = dw.shared = dx != nullptr;
    return dw.problems ? ffn_product(f, dw, s) : kOk;
}

int tgemm_ffn_get_kernels(tgemm_ffn_t f, int64_t tokens, tgemm_ffn_kernel_info *info)
{
    if (!f || !info || tokens < 1 || tokens > kMaxTokens) return kErrInvalidArg;
    const int64_t D = f->width, F = f->hidden, T = tokens;
    const Mat TF{nullptr, T, F, F}, TD{nullptr, T, D, D}, FD{nullptr, F, D, D}, DF{nullptr, D, F, F};
    // as the forward and the backward pass make them
    Job jobs[5] = {{kUp, 1, D, 1, 2, 3, {}, {}, {TF, TF, TF}},
                   {kDown, 1, F, 1, 1, 1, {}, {}, {TD}},
                   {kDh, 1, D, 1, 1, 2, {}, {}, {TF, TF}},
                   {kDx, 1, F, 2, 2, 1, {}, {}, {TD}},
                   {kDw, 3, T, 3, 3, 3, {}, {}, {FD, FD, DF}}};
    jobs[kDx].shared = jobs[kDw].shared = jobs[kDw].beside = true;
    for (int i = 0; i < 5; ++i) {
        const Cut c = ffn_cut(f, jobs[i]);
        info[i].kernel = c.few ? TGEMM_FFN_FEW : TGEMM_FFN_PAIRS;
        info[i].cluster = c.few ? c.shape.ranks : 2;
        if (i <= kDown && ffn_takes_rows(f, tokens)) {
            info[i].kernel = TGEMM_FFN_ROWS;
            info[i].cluster = 1;
        }
    }
    return kOk;
}

int tgemm_ffn_status(tgemm_ffn_t f, int *detail)
{
    if (!f) return kErrInvalidArg;
    int h[4] = {0, 0, 0, 0};
    if (cudaMemcpy(h, f->d_status, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(f->d_status, 0, sizeof(h)) != cudaSuccess) {
        cudaGetLastError();
        return -kErrCuda;
    }
    if (detail) std::memcpy(detail, h, sizeof(h));
    return h[0];
}

int tgemm_ffn_set_watchdog_ns(tgemm_ffn_t f, uint64_t ns)
{
    if (!f) return kErrInvalidArg;
    f->watchdog_ns = ns ? (unsigned long long)ns : env_watchdog();
    return kOk;
}

int tgemm_ffn_debug_stall(tgemm_ffn_t f, int on)
{
    if (!f) return kErrInvalidArg;
    f->debug_stall = on ? 1 : 0;
    return kOk;
}

int tgemm_ffn_destroy(tgemm_ffn_t f)
{
    if (!f) return kOk;
    const OutsideCapture relaxed;
    int rc = kOk;
    if (f->d_status && cudaFree(f->d_status) != cudaSuccess) {
        cudaGetLastError();
        rc = kErrCuda;
    }
    delete f;
    return rc;
}

}  // extern "C"
