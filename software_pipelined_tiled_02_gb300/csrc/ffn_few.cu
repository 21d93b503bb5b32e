// ffn_few.cu -- the feed-forward block's products with few tokens, for GB300
// (sm_103a).
//
// With few tokens the products are bound by streaming the weights.  The tiled
// kernel of ffn.cu would fill 256 tile rows with tokens and leave most SMs
// without a tile; here the weights are the MMA's 128 rows and the tokens its
// columns, and a tile's K range is shared out over a cluster of CTAs:
//   Up    64 hidden units: rows 0-63 are gate rows, 64-127 the units' up rows
//   Down, Dh, Dx   128 output features (Dh and Dx read the weights MN-major)
//   Dw    128 columns of a weight gradient; the MMA's columns are its rows, and
//         the sum runs over the tokens: for many tokens and small weights,
//         where whole tiles would leave most SMs idle
// Each CTA runs TMA -> ring -> tcgen05.mma over its K range into tensor memory.
// Then rank r of the cluster takes a slice of the tokens: every CTA writes its
// partial sums of that slice into r's shared memory (the ring is idle by then),
// and r adds them in rank order, applies what the product asks for and stores.
// The order of every sum is fixed by the sizes.
//
// One token, 4096 x 8192 bf16: 39 us forward, the weights' 201 MB at 5.2
// TB/s (Up alone 29 us, Down 19; Down's first weights load while Up ends).  64
// tokens: 43 us.  24 tokens, 512 x 2048: 9 us, two launches' latency.
//
// Two CTAs share an SM where their rings fit, so that one streams while the
// other reduces.  A product whose weights no preceding kernel of the call
// writes (Down, Dx) loads its first weight tiles while that kernel finishes.

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <type_traits>

#include "elem.cuh"
#include "ffn.cuh"
#include "host.h"
#include "layout.h"
#include "ptx.cuh"
#include "watchdog.cuh"

namespace tg {

constexpr int kFewThreads = 320;  // warp 0 loads, warp 1 issues MMAs, warps 2-9 read tensor memory
constexpr int kFewMaxStages = 8;

struct FewParams {  // 64-byte aligned through its CUtensorMap members
    CUtensorMap tmA[3], tmB[3];  // Up: gate and up weights; Dx: by K segment; Dw: by problem
    int problems;                // 1; Dw: up to 3 outputs
    int first_tile[4];           // of each problem, then the total
    int tokens[3], features[3];  // rows and columns of the output; Up: hidden units
    int token_tiles[3];          // tiles of n rows
    int n;                       // MMA columns: the tokens of a tile, a multiple of 16
    int num_kb, seg_kb;          // 64-element K blocks, and those of Dx's first segment
    int kb_each;                 // K blocks per rank of the cluster
    int ranks, slice;            // CTAs of a cluster, tokens of a rank's slice
    int stages;
    uint32_t slot, off_bar;      // bytes of a ring slot (A, then B), offset of the barriers
    int tmem_cols;
    uint32_t idesc;
    int early;                   // weights may be loaded before the preceding kernel has finished
    int beside;                  // Dw: see Job
    int bf16, act;
    void *out[3];                // Up: h, g, u (g and u may be NULL); Dh: dg, du; else by problem
    const void *g, *u;           // Dh
    int64_t ld_out[3];           // by problem
    unsigned long long watchdog_ns;
    int *status;
    int debug_stall;
};

template <int PROD>
__global__ void __launch_bounds__(kFewThreads) ffn_few_kernel(const __grid_constant__ FewParams p)
{
    constexpr bool A_MN = PROD == kDh || PROD == kDx || PROD == kDw, B_MN = PROD == kDw;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = (kSmemAlign - (raw & (kSmemAlign - 1))) & (kSmemAlign - 1);
    uint8_t *smem = smem_raw + pad;
    const uint32_t ring = raw + pad, bars = ring + p.off_bar;
    auto full = [&](int s) { return bars + 8u * uint32_t(s); };
    auto empty = [&](int s) { return bars + 8u * uint32_t(kFewMaxStages + s); };
    const uint32_t acc_full = bars + 8u * uint32_t(2 * kFewMaxStages), drain = acc_full + 8u, stall = acc_full + 16u;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + p.off_bar + 8u * (2 * kFewMaxStages + 3));
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32;
    const int rank = int(cluster_ctarank());
    constexpr int kTileRows = PROD == kUp ? 64 : 128;
    const int tile = int(blockIdx.x) / p.ranks;
    int prob = 0;
    if (PROD == kDw)
        while (prob + 1 < p.problems && tile >= p.first_tile[prob + 1]) ++prob;
    const int in_prob = tile - p.first_tile[prob];
    const int f0 = in_prob / p.token_tiles[prob] * kTileRows;  // the tile's first output feature and token
    const int token0 = in_prob % p.token_tiles[prob] * p.n;
    const int kb0 = min(rank * p.kb_each, p.num_kb), kb1 = min(kb0 + p.kb_each, p.num_kb);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(drain, 1);
        mbar_init(stall, 1);
        *abort = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tmA[0]);
        prefetch_tmap(&p.tmB[0]);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), uint32_t(p.tmem_cols));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Every thread waits here for the preceding kernel but the loading one, which
    // may start on weights first.
    const bool loader = warp == 0 && lane == 0;
    const bool beside = PROD == kDw && p.beside;
    if (!(loader && p.early) && !beside) griddep_wait();
    if (!loader) griddep_launch_dependents();

    int issued = 0;  // the loading thread's K blocks
    if (loader) {
        const int panels = (p.n + 63) / 64;  // MN-major B: boxes of 64 columns
        const uint32_t b_bytes = B_MN ? uint32_t(panels) * kPanel : uint32_t(p.n) * 128u;
        auto load_a = [&](int s, int kb) {
            const int seg = PROD == kDw ? prob : PROD == kDx && kb >= p.seg_kb ? 1 : 0;
            const int k = (kb - (PROD == kDx && seg ? p.seg_kb : 0)) * kBlockK;
            const uint32_t dst = ring + uint32_t(s) * p.slot;
            if constexpr (PROD == kUp) {
                tma_load_2d(dst, &p.tmA[0], k, f0, full(s));
                tma_load_2d(dst + kSlot / 2, &p.tmA[1], k, f0, full(s));
            } else if constexpr (A_MN) {
                tma_load_2d(dst, &p.tmA[seg], f0, k, full(s));
                tma_load_2d(dst + kPanel, &p.tmA[seg], f0 + 64, k, full(s));
            } else {
                tma_load_2d(dst, &p.tmA[0], k, f0, full(s));
            }
        };
        auto load_b = [&](int s, int kb) {
            const int seg = PROD == kDw ? prob : PROD == kDx && kb >= p.seg_kb ? 1 : 0;
            const int k = (kb - (PROD == kDx && seg ? p.seg_kb : 0)) * kBlockK;
            const uint32_t dst = ring + uint32_t(s) * p.slot + kSlot;
            if constexpr (B_MN) {
                for (int i = 0; i < panels; ++i)
                    tma_load_2d(dst + uint32_t(i) * kPanel, &p.tmB[seg], token0 + i * 64, k, full(s));
            } else {
                tma_load_2d(dst, &p.tmB[seg], k, token0, full(s));
            }
        };
        const int blocks = kb1 - kb0;
        const int first = blocks < p.stages ? blocks : p.stages;
        for (int i = 0; i < first; ++i) {
            mbar_arrive_expect_tx(full(i), kSlot + b_bytes);
            load_a(i, kb0 + i);
        }
        if (p.early) griddep_wait();
        griddep_launch_dependents();
        for (int i = 0; i < first; ++i) load_b(i, kb0 + i);
        int s = 0;
        uint32_t ph = 0;
        for (issued = first; issued < blocks; ++issued) {
            if (!mbar_try_wait(empty(s), ph) && !wait_bar(empty(s), ph, p, abort, 0, issued)) break;
            mbar_arrive_expect_tx(full(s), kSlot + b_bytes);
            load_a(s, kb0 + issued);
            load_b(s, kb0 + issued);
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
    } else if (warp == 1) {
        const uint64_t ad0 = ffn_desc(ring, A_MN), bd0 = ffn_desc(ring + kSlot, B_MN);
        constexpr uint64_t a_step = A_MN ? 2048 >> 4 : 32 >> 4, b_step = B_MN ? 2048 >> 4 : 32 >> 4;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        if (p.debug_stall) ok = warp_wait(stall, 0, p, abort, 1, 0);  // test hook: nothing arrives
        for (int kb = kb0; ok && kb < kb1; ++kb) {
            if (!warp_wait(full(s), ph, p, abort, 1, kb)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t at = uint64_t(s) * (p.slot >> 4);
            if (check(s < p.stages && kb < p.num_kb && p.n <= p.tmem_cols, p, abort, 1, kb)) {
#pragma unroll
                for (int kk = 0; kk < kBlockK / 16; ++kk)
                    mma_f16(tmem, ad0 + at + uint64_t(kk) * a_step, bd0 + at + uint64_t(kk) * b_step, p.idesc,
                            kk || kb > kb0 ? 1u : 0u);
            }
            mma_commit_elect(empty(s));
            __syncwarp();
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (ok && kb0 < kb1) mma_commit_elect(acc_full);
        __syncwarp();
        if (lane == 0) {  // every MMA issued has to finish before the ring is reused and TMEM freed
            mma_commit(drain);
            wait_bar(drain, 0, p, abort, 1, kb1, false);
        }
    }
    __syncwarp();
    // Partial sums: warp w reads TMEM lanes 32 (w % 4) .. + 31, one weight row a
    // lane; the two warps of a quarter take a half of the tokens' 16-column chunks
    // each.
    const bool reader = warp >= 2;
    const int row = (warp & 3) * 32 + lane;
    const bool have = reader && kb0 < kb1 && warp_wait(acc_full, 0, p, abort, 2, 0);
    tc_fence_after();
    __syncwarp();
    cluster_sync();  // every ring of the cluster is idle
    if (loader && *abort) {  // nothing may have waited for the last loads: they land before the CTA exits
        for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
            wait_bar(full(i % p.stages), uint32_t(i / p.stages) & 1u, p, abort, 0, i, false);
    }
    __syncwarp();
    // Rank r's slice: partial sums [rank][token / 4][row][token % 4], so that a
    // warp writes and reads 512 bytes on end.
    const uint32_t region = uint32_t(p.slice) * 512u;
    if (reader && !*abort) {
        // Tokens in order, four at a time, so that owner and place in its slice only step on.
        const int half = (p.n / 16 + 1) / 2 * 16;
        const int begin = warp < 6 ? 0 : half, end = warp < 6 ? half : p.n;
        int owner = begin / p.slice, in = begin - owner * p.slice;
        const uint32_t mine = ring + uint32_t(rank) * region + uint32_t(row) * 16u;
        uint32_t at = map_to_rank(mine, uint32_t(owner < p.ranks ? owner : 0)) + uint32_t(in) * 512u;
        for (int t0 = begin; t0 < end; t0 += 16) {
            uint32_t v[16];
            if (have) {
                asm volatile(
                    "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                    "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                    : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                      "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                      "=r"(v[15])
                    : "r"(tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(t0))
                    : "memory");
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0u;  // no K block fell to this rank
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                if (check(owner < p.ranks && in + 4 <= p.slice && uint32_t(rank + 1) * region <= p.off_bar, p, abort, 2, t0))
                    st_cluster_v4(at, v[e], v[e + 1], v[e + 2], v[e + 3]);
                at += 2048;
                in += 4;
                if (in == p.slice) {
                    in = 0;
                    at = map_to_rank(mine, uint32_t(++owner < p.ranks ? owner : 0));
                }
            }
        }
    }
    tc_fence_before();
    cluster_sync();  // the slices are complete
    if (!*abort) {
        // One feature and four tokens a thread: sums over the ranks in rank order.
        const int first = token0 + rank * p.slice;  // the slice's first token
        const int tokens = min(p.slice, min(p.n - rank * p.slice, p.tokens[prob] - first));  // of it that exist
        const int rows = min(kTileRows, p.features[prob] - f0);
        auto item = [&](auto act_c, int i) {
            constexpr int ACT = decltype(act_c)::value;
            const int t = i / kTileRows * 4, r = i % kTileRows;
            if (r >= rows) return;
            const int count = min(4, tokens - t);
            const int64_t o = int64_t(first + t) * p.ld_out[prob] + f0 + r;
            uint16_t gw[4] = {}, uw[4] = {};
            if constexpr (PROD == kDh) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e >= count) break;
                    gw[e] = static_cast<const uint16_t *>(p.g)[o + e * p.ld_out[prob]];
                    uw[e] = static_cast<const uint16_t *>(p.u)[o + e * p.ld_out[prob]];
                }
            }
            uint32_t at = ring + uint32_t(t) * 512u + uint32_t(r) * 16u;
            F2 s[2] = {f2(0.f), f2(0.f)}, s_up[2] = {f2(0.f), f2(0.f)};
            for (int q = 0; q < p.ranks; ++q, at += region) {
                const float4 v = ld_shared_v4f(at);
                s[0] = s[0] + f2(v.x, v.y);
                s[1] = s[1] + f2(v.z, v.w);
                if constexpr (PROD == kUp) {
                    const float4 w = ld_shared_v4f(at + 64u * 16u);
                    s_up[0] = s_up[0] + f2(w.x, w.y);
                    s_up[1] = s_up[1] + f2(w.z, w.w);
                }
            }
            auto put = [&](int which, const F2 (&v)[2]) {
                const uint32_t w[2] = {pack2(v[0], p.bf16), pack2(v[1], p.bf16)};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < count && check(first + t + e < p.tokens[prob] && f0 + r < p.features[prob], p, abort, 2, t))
                        static_cast<uint16_t *>(p.out[which])[o + e * p.ld_out[prob]] = uint16_t(w[e / 2] >> (e % 2 * 16));
            };
            if constexpr (PROD == kUp) {
                F2 h[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    F2 act, slope;
                    activate<ACT>(s[e], act, slope);
                    h[e] = act * s_up[e];
                }
                put(0, h);
                if (p.out[1]) {
                    put(1, s);
                    put(2, s_up);
                }
            } else if constexpr (PROD == kDh) {
                F2 dg[2], du[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 g = unpack2(gw[2 * e] | uint32_t(gw[2 * e + 1]) << 16, p.bf16);
                    const float2 u = unpack2(uw[2 * e] | uint32_t(uw[2 * e + 1]) << 16, p.bf16);
                    F2 act, slope;
                    activate<ACT>(f2(g.x, g.y), act, slope);
                    dg[e] = s[e] * f2(u.x, u.y) * slope;
                    du[e] = s[e] * act;
                }
                put(0, dg);
                put(1, du);
            } else {
                put(PROD == kDw ? prob : 0, s);
            }
        };
        auto items = [&](auto act_c) {
            const int count = (tokens + 3) / 4 * kTileRows;  // none where the slice lies past the tokens
            for (int i = int(threadIdx.x); i < count; i += kFewThreads) item(act_c, i);
        };
        if ((PROD != kUp && PROD != kDh) || p.act == kSilu)
            items(std::integral_constant<int, kSilu>{});
        else if (p.act == kGelu)
            items(std::integral_constant<int, kGelu>{});
        else
            items(std::integral_constant<int, kRelu>{});
    }
    if (beside) griddep_wait();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, uint32_t(p.tmem_cols));
    }
}

// ---------------------------------------------------------------- host side

typedef void (*FewKernel)(const FewParams);
static const FewKernel kFewKernels[5] = {ffn_few_kernel<kUp>, ffn_few_kernel<kDown>, ffn_few_kernel<kDh>,
                                         ffn_few_kernel<kDx>, ffn_few_kernel<kDw>};

static int few_setup(const Device &d)
{
    static std::atomic<uint64_t> done{0};
    if (d.ordinal < 64 && (done.load() >> d.ordinal & 1)) return kOk;
    for (FewKernel k : kFewKernels) {
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem_limit) != cudaSuccess ||
            cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return kErrCuda;
        }
    }
    if (d.ordinal < 64) done.fetch_or(uint64_t(1) << d.ordinal);
    return kOk;
}

// Tokens of a rank's slice: a multiple of 4.
static int few_slice(int n, int ranks) { return ((n + ranks - 1) / ranks + 3) / 4 * 4; }

// Bytes of the partial sums in a CTA's shared memory (the kernel's `region`s).
static uint32_t few_sums_bytes(int n, int ranks)
{
    return uint32_t(ranks) * uint32_t(few_slice(n, ranks)) * 512u;
}

// The ring with two CTAs on an SM: bytes of a slot, slots, and bytes in all.
constexpr uint32_t kFewBarBytes = 8 * (2 * kFewMaxStages + 3) + 16 + kSmemAlign;
static uint32_t few_slot_bytes(const Job &j, int n)
{
    return kSlot + uint32_t(j.prod == kDw ? (n + 63) / 64 * 64 : n) * 128u;
}
static int few_stages(const tgemm_ffn_s *f, const Job &j, int n)
{
    const int fit = int((uint32_t(f->dev.smem_per_sm) / 2 - 1024 - kFewBarBytes) / few_slot_bytes(j, n));
    return fit < kFewMaxStages ? fit : kFewMaxStages;
}
static uint32_t few_ring_bytes(const tgemm_ffn_s *f, const Job &j, int n)
{
    return uint32_t(few_stages(f, j, n)) * few_slot_bytes(j, n);
}

// The shape with the fewest estimated SM cycles among clusters of 1 to 16 CTAs
// and token tiles of 16 to 128 columns.  For each round of CTAs:
//  * a K block: its operands at 64 bytes a cycle from L2 (the MMAs take 2 n),
//    shared by the CTAs of an SM, but not less than a ring's latency, about 2850,
//    over its slots;
//  * the partial sums' way out, 32 a token, and through the cluster first, 16,
//    both shared by the CTAs of an SM;
//  * 10000 for set-up and hand-overs, 1200 more for a cluster of 16.
// Dx and Dw add their share of the machine.
// How the constants were found stands at tile_width in ffn.cu.
FewShape ffn_few_shape(const tgemm_ffn_s *f, const Job &j, double *cycles)
{
    FewShape best{};
    const int64_t sms = f->dev.sms;
    const int tile_rows = j.prod == kUp ? 64 : 128;
    const int64_t seg_kb = (j.k + kBlockK - 1) / kBlockK, num_kb = j.prod == kDx ? 2 * seg_kb : seg_kb;
    int64_t most = 0;  // rows of the tallest output
    for (int i = 0; i < j.problems; ++i) most = j.C[i].rows > most ? j.C[i].rows : most;
    *cycles = 0.0;
    // Up to 128 columns, two CTAs an SM have a ring of three slots or more each.
    for (int64_t token_tiles = (most + 127) / 128;; token_tiles *= 2) {
        const int64_t n = ((most + token_tiles - 1) / token_tiles + 15) / 16 * 16;
        int64_t tiles = 0;
        for (int i = 0; i < j.problems; ++i)
            tiles += (j.C[i].cols + tile_rows - 1) / tile_rows * ((j.C[i].rows + n - 1) / n);
        const double slot = 2850.0 / few_stages(f, j, int(n));
        for (int ranks = 1; ranks <= 16; ranks *= 2) {
            // an SM's two CTAs; clusters of 8 and 16 leave some SMs of a group unused
            const int64_t room = ranks < 8 ? 2 * sms : ranks == 8 ? 2 * sms * 15 / 16 : 2 * sms * 11 / 16;
            if (ranks > 1 && (tiles * ranks > room || num_kb < 2 * ranks ||
                              few_sums_bytes(int(n), ranks) > few_ring_bytes(f, j, int(n))))
                break;
            const int64_t rounds = (tiles * ranks + room - 1) / room, kb_each = (num_kb + ranks - 1) / ranks;
            const double together = tiles * ranks > sms ? 2.0 : 1.0, feed = together * (256.0 + 2.0 * double(n));
            const double out = together * double(n) * (32.0 + 16.0 * (ranks - 1) / ranks);
            const double round = double(kb_each) * (feed > slot ? feed : slot) + out +
                                 (ranks == 16 ? 11200.0 : 10000.0);
            double c = double(rounds) * round;
            if (j.shared) c += kShare * double(tiles * ranks) * round / double(2 * sms);
            if (*cycles == 0.0 || c < *cycles) {
                *cycles = c;
                best.tiles = tiles;
                best.ranks = ranks;
                best.n = int(n);
                best.kb_each = int(kb_each);
            }
        }
        if (n == 16) break;
    }
    return best;
}

int ffn_few_product(tgemm_ffn_s *f, const Job &j, const FewShape &c, cudaStream_t s)
{
    const bool up = j.prod == kUp, a_mn = j.prod == kDh || j.prod == kDx || j.prod == kDw, b_mn = j.prod == kDw;
    int rc = few_setup(f->dev);
    if (rc != kOk) return rc;
    if (c.tiles * c.ranks > (int64_t(1) << 30)) return kErrInvalidArg;
    FewParams p;
    std::memset(&p, 0, sizeof(p));
    p.problems = j.problems;
    p.seg_kb = int((j.k + kBlockK - 1) / kBlockK);
    p.num_kb = j.prod == kDx ? 2 * p.seg_kb : p.seg_kb;
    p.ranks = c.ranks;
    p.n = c.n;
    const int tile_rows = up ? 64 : 128;
    for (int i = 0, total = 0; i < j.problems; ++i) {
        p.tokens[i] = int(j.C[i].rows);
        p.features[i] = int(j.C[i].cols);
        p.token_tiles[i] = (p.tokens[i] + p.n - 1) / p.n;
        p.ld_out[i] = j.C[i].ld;
        p.first_tile[i] = total;
        total += (p.features[i] + tile_rows - 1) / tile_rows * p.token_tiles[i];
    }
    p.slot = few_slot_bytes(j, p.n);
    p.stages = few_stages(f, j, p.n);
    p.kb_each = c.kb_each;
    p.slice = few_slice(p.n, p.ranks);
    if (p.stages < 1 || few_sums_bytes(p.n, p.ranks) > uint32_t(p.stages) * p.slot) return kErrSmemBudget;
    p.off_bar = uint32_t(p.stages) * p.slot;
    const uint32_t smem = p.off_bar + kFewBarBytes;
    p.tmem_cols = 32;
    while (p.tmem_cols < p.n) p.tmem_cols *= 2;
    // Instruction descriptor (layout as in tgemm.cu): M = 128, N = n, bits 15
    // and 16 mark MN-major A and B.
    const uint32_t ab = f->dtype == kBF16 ? 1u : 0u;
    p.idesc = (1u << 4) | (ab << 7) | (ab << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
              (uint32_t(p.n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    // The weights are the job's B, the tokens its A.
    const int weights = up || j.prod == kDx ? 2 : j.problems, tokens = j.prod == kDx ? 2 : j.problems;
    for (int i = 0; i < weights && rc == kOk; ++i) {
        const Mat &w = j.B[i];
        const uint64_t pitch = uint64_t(w.ld) * 2;
        rc = encode_2d(&p.tmA[i], f->dtype, w.p, uint64_t(w.cols), uint64_t(w.rows), pitch, 64, up || a_mn ? 64 : 128,
                       CU_TENSOR_MAP_SWIZZLE_128B, operand_promotion(pitch));
    }
    for (int i = 0; i < tokens && rc == kOk; ++i) {
        const Mat &x = j.A[i];
        const uint64_t pitch = uint64_t(x.ld) * 2;
        rc = encode_2d(&p.tmB[i], f->dtype, x.p, uint64_t(x.cols), uint64_t(x.rows), pitch, 64, b_mn ? 64u : uint32_t(p.n),
                       CU_TENSOR_MAP_SWIZZLE_128B, operand_promotion(pitch));
    }
    if (rc != kOk) return rc;
    p.early = j.prod == kDown || j.prod == kDx;
    p.beside = j.beside;
    p.bf16 = f->dtype == kBF16;
    p.act = f->act;
    for (int i = 0; i < j.nc; ++i) p.out[i] = const_cast<void *>(j.C[i].p);
    p.g = j.g;
    p.u = j.u;
    p.watchdog_ns = f->watchdog_ns;
    p.status = f->d_status;
    p.debug_stall = f->debug_stall;
    return launch(kFewKernels[j.prod], dim3(unsigned(c.tiles * p.ranks)), dim3(kFewThreads), smem, s, unsigned(p.ranks), p);
}

}  // namespace tg
