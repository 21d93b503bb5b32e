// experts_few.cu -- the experts' feed-forward blocks for a few tokens, for GB300
// (sm_103a).
//
// With a few pairs of a token and an expert the pass is the stream of the chosen
// experts' weights, and ordering pairs, gathering rows and filling 256-row tiles
// would only come before it.  Here a CTA finds its experts and these experts' pairs
// itself, from the list of choices, and the weights go from memory straight into
// the registers of tensor-core fragments (as in ffn_rows.cu): 16 weight rows, 8
// pairs, and k shared out among the CTA's warps.  Three launches:
//   up       h, 8 hidden units a block: rows 0-7 are gate rows, 8-15 the same units' up rows
//   down     each pair's result, 16 features a block, in fp32; its first weights are on
//            their way while up ends
//   combine  each token's weighted sum (experts_rows.cu); for one token `down` adds
//            its experts' results itself
// Rows of h and of down's results are numbered by pair.
//
// What bounds it: the weights' stream, with three (two) launches' latency before and
// after.  One token, 8 of 64 experts of 2048 x 1024 bf16 (101 MB): 22.8 us, 4.4 TB/s;
// 2 of 32 of 4096 x 1536 (75 MB): 17.2; 8 tokens of the latter 76 to 84 us, 6.1 TB/s.  Against
// the ordered way: 16 tokens, 8 of 64 of 2048 x 1408 156 us and 200; 24 tokens, 6 of 64
// of 1024 x 512 42 and 55; 16 tokens, 4 of 16 of 2048 x 1408 48 and 71; where an expert
// has more than 8 pairs 202 and 158 (32 tokens, 2 of 8 of 4096 x 4096), which
// experts_are_few() therefore leaves to it; 64 tokens, 8 of 128 of 1024 x 512 (512
// pairs) 94 and 94.  A grid cut for as many experts as alike choices would name took 61
// us where 8 tokens chose the same 8 of 64 of 2048 x 1408, and this one 34; 8 tokens, 6
// of 64 of 1024 x 512 with choices that differ take 27.6 instead of 26.  Blocks of rows
// one after the other in the same CTA, the next one's weights on their way while the
// last one's sums are added, measured 22.6 us (one token) where a CTA for each block
// took 27.9.  16 pairs at a time (two steps for each weight fragment) were slower than
// this and than whole tiles: 348 us against 204 (48 tokens, 4 of 32).

#include <algorithm>
#include <cmath>

#include "elem.cuh"
#include "experts.cuh"
#include "ffn.cuh"
#include "host.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace tg {

constexpr int kFewWarps = 8;
constexpr int kFewChunk = 128;  // k per warp and step: four 16-byte loads a lane and weight row
constexpr int kFewAhead = 2;    // steps whose weights are on their way

struct ExpertsFew {
    Pairs pairs;
    int top;
    int64_t width, hidden, ldx;
    const uint16_t *x;
    const uint16_t *w[3];  // gate, up, down
    int64_t ld[3], es[3];
    uint16_t *h;           // [pairs][hidden]
    float *y;              // [pairs][width]
    int act;
};

// 16 bytes of a weight, which is not read again: kept out of L1.
__device__ __forceinline__ uint4 load_weights16(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The blocks of rows of all experts that a pair names are shared out evenly among the
// CTAs, which find these experts themselves: how many there are is known here alone.
// ONE: a single token's `up`, where the host knows it and blockIdx.y is the slot; finding
// the experts would take 1 us of its 20.
// A CTA's warps walk through its blocks' steps without a pause: the next block's first
// weights are on their way while this one's sums are added, by one warp, from one of
// two sets.
template <bool BF16, bool UP, bool ONE>
__global__ void __launch_bounds__(32 * kFewWarps, 2) experts_few_kernel(const ExpertsFew a)
{
    __shared__ float4 part[2][kFewWarps][32];
    __shared__ int list[8], listed[2], first_pair[kMostExperts], named[kFewPairs], num_named;
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32, g = lane / 4, c = lane % 4;
    if (UP) griddep_wait();
    griddep_launch_dependents();
    // The choices were there before `up` began, and so were the weights.
    int expert = 0;
    if constexpr (ONE) {
        static_assert(UP, "experts_one_kernel takes down");
        if (!slot_expert(a.pairs, int(blockIdx.y), expert) || expert < 0) return;
    }
    // The experts that pairs name, in the order of their first pairs.
    if (!ONE && a.pairs.pairs > 32) {
        for (int e = int(threadIdx.x); e < a.pairs.num_experts; e += 32 * kFewWarps) first_pair[e] = a.pairs.pairs;
        __syncthreads();
        for (int i = int(threadIdx.x); i < a.pairs.pairs; i += 32 * kFewWarps) {
            const int e = expert_of(a.pairs, i);
            if (e >= 0) atomicMin(&first_pair[e], i);
        }
        __syncthreads();
    }
    if (!ONE && warp == 0) {
        int n = 0;
        for (int i0 = 0; i0 < a.pairs.pairs; i0 += 32) {
            const int e = i0 + lane < a.pairs.pairs ? expert_of(a.pairs, i0 + lane) : -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const bool first = e >= 0 && (a.pairs.pairs > 32 ? first_pair[e] == i0 + lane : __ffs(int(same)) - 1 == lane);
            const unsigned found = __ballot_sync(0xffffffffu, first);
            if (first) named[n + __popc(found & ((1u << lane) - 1u))] = e;
            n += __popc(found);
        }
        if (lane == 0) num_named = n;
    }
    if (!ONE) __syncthreads();
    constexpr int kBlock = UP ? 8 : 16;  // hidden units or features
    const int K = int(UP ? a.width : a.hidden), N = int(UP ? a.hidden : a.width), blocks = (N + kBlock - 1) / kBlock;
    const int steps = max(0, (K + kFewChunk - 1 - warp * kFewChunk) / kFewChunk + kFewWarps - 1) / kFewWarps;  // of this warp, a block
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const int64_t all = ONE ? blocks : int64_t(num_named) * blocks, end = all * (blockIdx.x + 1) / gridDim.x;
    int64_t unit = all * blockIdx.x / gridDim.x;
    int last = 0;  // the block behind the expert's last one here
    uint4 wl[kFewAhead][4], wh[kFewAhead][4];
    // The weights that come next.
    int next_block = 0, next_step = 0;
    const uint16_t *lo = nullptr, *hi = nullptr;
    bool high = false;
    auto start_block = [&](int block) {
        next_block = block;
        next_step = 0;
        const int64_t row = int64_t(block) * kBlock + g;  // of the low half; hidden and width are multiples of 8
        const int64_t k = warp * kFewChunk + c * 8;
        lo = a.w[UP ? 0 : 2] + expert * a.es[UP ? 0 : 2] + row * a.ld[UP ? 0 : 2] + k;
        hi = UP ? a.w[1] + expert * a.es[1] + row * a.ld[1] + k : lo + 8 * a.ld[2];
        high = UP || row + 8 < N;
    };
    auto load = [&](int s) {
        if (next_block >= last || steps == 0) return;
        const int left = K - (warp + next_step * kFewWarps) * kFewChunk - c * 8;  // of this lane's row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wl[s][i] = i * 32 < left ? load_weights16(lo + i * 32) : none;
            wh[s][i] = i * 32 < left && high ? load_weights16(hi + i * 32) : none;
        }
        lo += kFewWarps * kFewChunk;
        hi += kFewWarps * kFewChunk;
        if (++next_step == steps) start_block(next_block + 1);
    };
    bool waited = UP;
    int from = 0, first = 0;
    for (bool turned = true; unit < end || !turned;) {
        if (turned) {  // the next expert's blocks
            const int n = ONE ? 0 : int(unit / blocks);
            if (!ONE) expert = named[n];
            first = int(unit - int64_t(n) * blocks);
            last = int(min(int64_t(blocks), first + end - unit));
            unit += last - first;
            from = 0;
        }
        start_block(first);
#pragma unroll
        for (int s = 0; s < kFewAhead; ++s) load(s);
        if (warp == 0) {
            int n;
            const int next = list_pairs(a.pairs, expert, from, 8, list, n);
            if (lane == 0) {
                listed[0] = n;
                listed[1] = next;
            }
        }
        if (!waited) griddep_wait();  // h is there
        waited = true;
        __syncthreads();
        const int count = listed[0];
        from = listed[1];
        if (count == 0) {  // 8 pairs were all
            turned = true;
            __syncthreads();
            continue;
        }
        // columns of pairs that are not there repeat the last one's and are dropped
        const int pair = list[min(g, count - 1)];
        const uint16_t *x = (UP ? a.x + int64_t(pair / a.top) * a.ldx : a.h + int64_t(pair) * a.hidden) + warp * kFewChunk + c * 8;
        float s[4] = {};
        int block = first, step = 0, turn = 0;
        auto close_block = [&] {  // the warps' sums of a block: added in warp order, and stored
            part[turn & 1][warp][lane] = make_float4(s[0], s[1], s[2], s[3]);
            s[0] = s[1] = s[2] = s[3] = 0.f;
            __syncthreads();
            if (turn % kFewWarps == warp) {
                float4 v = part[turn & 1][0][lane];
#pragma unroll
                for (int w = 1; w < kFewWarps; ++w) {
                    const float4 q = part[turn & 1][w][lane];
                    v.x += q.x;
                    v.y += q.y;
                    v.z += q.z;
                    v.w += q.w;
                }
                const int64_t row = int64_t(block) * kBlock + g;
                // columns 2 c and 2 c + 1: (gate x, up z), (gate y, up w), or two features
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (c * 2 + e >= count) continue;
                    const int64_t to = list[c * 2 + e];
                    const float low = e ? v.y : v.x, upper = e ? v.w : v.z;
                    if constexpr (UP) {
                        float act, slope;
                        if (a.act == kSilu)
                            activate<kSilu>(low, act, slope);
                        else if (a.act == kGelu)
                            activate<kGelu>(low, act, slope);
                        else
                            activate<kRelu>(low, act, slope);
                        a.h[to * a.hidden + row] = uint16_t(pack2(act * upper, 0.f, BF16));
                    } else {
                        a.y[to * a.width + row] = low;
                        if (row + 8 < N) a.y[to * a.width + row + 8] = upper;
                    }
                }
            }
            ++block;
            step = 0;
            ++turn;
        };
        if (steps == 0) {  // few k: this warp has none of them
            while (block < last) close_block();
        }
        while (block < last) {
#pragma unroll
            for (int u = 0; u < kFewAhead; ++u) {
                if (block >= last) break;
                const int left = K - (warp + step * kFewWarps) * kFewChunk - c * 8;
                const uint16_t *at = x + step * (kFewWarps * kFewChunk);
                uint4 t[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = i * 32 < left ? *reinterpret_cast<const uint4 *>(at + i * 32) : none;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_few<BF16>(s, wl[u][i].x, wh[u][i].x, wl[u][i].y, wh[u][i].y, t[i].x, t[i].y);
                    mma_few<BF16>(s, wl[u][i].z, wh[u][i].z, wl[u][i].w, wh[u][i].w, t[i].z, t[i].w);
                }
                load(u);
                if (++step == steps) close_block();
            }
        }
        turned = from >= a.pairs.pairs;
        __syncthreads();  // the sums and the list are read
    }
    if (!waited) griddep_wait();
}

// `down` and the weighted sum of a single token: a CTA takes 16 features, and its
// warps the token's experts in turn, one or several of them for each expert's k.
template <bool BF16>
__global__ void __launch_bounds__(32 * kFewWarps, 2) experts_one_kernel(const ExpertsFew a, const float *weights, uint16_t *y)
{
    __shared__ float part[kFewWarps][16];
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32, g = lane / 4, c = lane % 4;
    griddep_launch_dependents();
    const int K = int(a.hidden), N = int(a.width), slices = max(1, kFewWarps / a.top), steps = (K + kFewChunk - 1) / kFewChunk;
    const int each = (steps + slices - 1) / slices, units = a.top * slices;  // steps of a unit: a slice of an expert's k
    const int64_t row = int64_t(blockIdx.x) * 16 + g;
    const bool high = row + 8 < N;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    float sum[2] = {0.f, 0.f};  // of features g and g + 8
    bool waited = false;
    for (int unit = warp; unit < units; unit += kFewWarps) {
        const int pair = unit / slices, first = unit % slices * each, last = min(first + each, steps);
        const int expert = expert_of(a.pairs, pair);
        if (expert < 0) continue;
        const uint16_t *lo = a.w[2] + expert * a.es[2] + row * a.ld[2] + c * 8, *hi = lo + 8 * a.ld[2];
        const uint16_t *x = a.h + int64_t(pair) * K + c * 8;
        uint4 wl[kFewAhead][4], wh[kFewAhead][4];
        auto load = [&](int s, int step) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = step * kFewChunk + i * 32;
                const bool in = step < last && k + c * 8 < K;
                wl[s][i] = in ? load_weights16(lo + k) : none;
                wh[s][i] = in && high ? load_weights16(hi + k) : none;
            }
        };
#pragma unroll
        for (int s = 0; s < kFewAhead; ++s) load(s, first + s);
        if (!waited) griddep_wait();  // h is there
        waited = true;
        float s[4] = {};
        for (int step0 = first; step0 < last; step0 += kFewAhead) {
#pragma unroll
            for (int u = 0; u < kFewAhead; ++u) {
                const int step = step0 + u;
                uint4 t[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = step * kFewChunk + i * 32;
                    t[i] = step < last && k + c * 8 < K ? *reinterpret_cast<const uint4 *>(x + k) : none;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_few<BF16>(s, wl[u][i].x, wh[u][i].x, wl[u][i].y, wh[u][i].y, t[i].x, t[i].y);
                    mma_few<BF16>(s, wl[u][i].z, wh[u][i].z, wl[u][i].w, wh[u][i].w, t[i].z, t[i].w);
                }
                load(u, step + kFewAhead);
            }
        }
        const float w = weights[pair];  // all columns are the token's
        sum[0] = fmaf(s[0], w, sum[0]);
        sum[1] = fmaf(s[2], w, sum[1]);
    }
    if (!waited) griddep_wait();
    if (c == 0) {
        part[warp][g] = sum[0];
        part[warp][g + 8] = sum[1];
    }
    __syncthreads();
    const int64_t feature = int64_t(blockIdx.x) * 16 + threadIdx.x;
    if (threadIdx.x < 16 && feature < N) {
        float v = part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kFewWarps; ++i) v += part[i][threadIdx.x];
        y[feature] = uint16_t(pack2(v, 0.f, BF16));
    }
}

// Experts that more than 8 of the tokens choose, were all experts liked alike.
static double experts_crowded(const ExpertSizes &z)
{
    if (z.top >= z.experts) return z.tokens > 8 ? double(z.experts) : 0.0;
    const double share = double(z.top) / double(z.experts);
    double p = std::pow(1.0 - share, double(z.tokens)), few = p;  // of j tokens
    for (int j = 0; j < 8; ++j) few += p *= double(z.tokens - j) / double(j + 1) * share / (1.0 - share);
    return double(z.experts) * (1.0 - few);
}

bool experts_are_few(const ExpertSizes &z) { return z.pairs <= kFewPairs && experts_crowded(z) < 0.4; }

int experts_few(const ExpertsFewCall &call, const Combine &combine, const ExpertSizes &z, int sms, bool bf16, cudaStream_t s)
{
    ExpertsFew a{};
    a.pairs = Pairs{call.chosen, int(z.pairs), int(z.experts)};
    a.top = z.top;
    a.width = call.width;
    a.hidden = call.hidden;
    a.ldx = call.ldx;
    a.x = static_cast<const uint16_t *>(call.x);
    for (int i = 0; i < 3; ++i) {
        a.w[i] = static_cast<const uint16_t *>(call.w[i]);
        a.ld[i] = call.ld[i];
        a.es[i] = call.es[i];
    }
    a.h = static_cast<uint16_t *>(call.h);
    a.y = const_cast<float *>(combine.rows);
    a.act = call.act;
    const int64_t room = int64_t(2) * sms;  // two CTAs an SM
    const dim3 block(32 * kFewWarps);
    int rc;
    if (z.tokens == 1) {
        // As many blocks for each CTA as for the others, all in one round.
        const int64_t slots = slots_of(a.pairs), units = a.hidden / 8, fit = std::max<int64_t>(1, room / slots);
        const int64_t each = (units + fit - 1) / fit;
        const dim3 up(unsigned((units + each - 1) / each), unsigned(slots));
        rc = bf16 ? launch(experts_few_kernel<true, true, true>, up, block, 0, s, 1, a)
                  : launch(experts_few_kernel<false, true, true>, up, block, 0, s, 1, a);
        if (rc != kOk) return rc;
        uint16_t *y = static_cast<uint16_t *>(combine.out);
        const dim3 features(unsigned((a.width + 15) / 16));
        return bf16 ? launch(experts_one_kernel<true>, features, block, 0, s, 1, a, combine.weights, y)
                    : launch(experts_one_kernel<false>, features, block, 0, s, 1, a, combine.weights, y);
    }
    const int64_t most = std::min<int64_t>(z.experts, z.pairs);
    const dim3 up(unsigned(std::min(most * (a.hidden / 8), room))), down(unsigned(std::min(most * ((a.width + 15) / 16), room)));
    rc = bf16 ? launch(experts_few_kernel<true, true, false>, up, block, 0, s, 1, a)
              : launch(experts_few_kernel<false, true, false>, up, block, 0, s, 1, a);
    if (rc != kOk) return rc;
    rc = bf16 ? launch(experts_few_kernel<true, false, false>, down, block, 0, s, 1, a)
              : launch(experts_few_kernel<false, false, false>, down, block, 0, s, 1, a);
    if (rc != kOk) return rc;
    Placed none{};
    Combine c = combine;
    c.chosen = call.chosen;
    c.experts = int(z.experts);
    return experts_combine(z, call.width, bf16, c, none, s);
}

}  // namespace tg
