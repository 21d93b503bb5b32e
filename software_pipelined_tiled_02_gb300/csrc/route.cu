// route.cu -- routing of tokens to experts, its gradient, and its C ABI.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),   key_e = s_e + bias_e
//   a group's score: the sum of its largest one or two keys
//   experts: the top k keys among the experts of the best groups, largest first,
//   ties to the lowest index;   w_j = scale s_j, or scale s_j / sum_i s_i
//
// One warp a token: lane i holds the experts i, i + 32, ...  The k rounds each
// take the largest key that is left: keys are mapped to unsigned integers of the
// same order, and two warp-wide integer reductions find the value and its lowest
// index.
//
// The order is that of the exact scores.  Without a bias (and without sums of
// two keys) that is the logits' own order, which takes no rounding.  With one,
// keys are formed in fp32, and where two neighbours in the result are nearer
// than their rounding errors can account for, the keys in question are formed
// again in 64 bits.
//
// What bounds it: instructions, a thousand or so a token, where its bytes take
// little.  8192 tokens, 256 experts, 8 chosen, fp32 (8.9 MB, 1.3 us at the memory's
// rate): 7.8 us; by sigmoid scores with a bias 10 to 11, with a bias and 4 of 8 groups 13
// to 14.9, by how many near ties there are, of which softmax has more (17 to 20, 19 to
// 24).  The rounds take 30 instructions each, the groups 400 in all, scores and near ties
// 160; every register of logits, keys and their best two stays in the warp (80 registers).
// Two tokens a warp would share the rounds' instructions, but not the reductions: the two
// integer ones work on whole warps.  32 tokens of 128 experts take 2.4 us, a launch's
// latency.  The gradient of 8192 x 64 takes 3.8 us, of 1001 x 100 2.3.

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"
#include "ffn.cuh"
#include "host.h"
#include "ptx.cuh"
#include "tgemm.h"

namespace tg {

constexpr int kRouteWarps = 4;
constexpr int kMaxExperts = 1024, kMaxTop = 32, kMaxGroups = 32;
constexpr unsigned kAll = 0xffffffffu;

struct Route {
    const void *logits;
    int64_t ld, tokens;
    const float *bias;
    float *weights;
    int *experts;
    int n, top, groups, top_groups, group_scores;
    bool sigmoid, renorm;
    unsigned inv_size;  // 2^20 over a group's size, rounded up: e * inv_size >> 20 is e's group
    bool score_groups;  // the groups' scores come from scores, not from logits
    float scale;
};

// fp32 values as unsigned integers of the same order: -0 as +0, every NaN (which
// the sum makes the positive canonical one) above all others, nothing below 1 (0
// stands for "no value").
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k ^ (~uint32_t(int32_t(k) >> 31) | 0x80000000u));
}
constexpr uint32_t kNan = 0xffffffffu;  // ordered(NaN)
__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) < INFINITY; }

__device__ __forceinline__ double warp_max(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

// sigmoid(l) exp(-shift), for shift = min(largest l, 0)
__device__ __forceinline__ float relative_sigmoid(float l, float shift)
{
    return expf(fminf(l, 0.f) - shift) / (1.f + expf(-fabsf(l)));
}

// Scores that only the order needs, with the hardware's exp2 (2^-22 relatively) and
// reciprocal (1 ulp).
__device__ __forceinline__ float quick_exp(float x) { return exp2_approx(x * 1.44269504088896341f); }
__device__ __forceinline__ float quick_score(float l, bool is_sigmoid, float top, float inv_total)
{
    if (is_sigmoid) return rcp_approx(1.f + quick_exp(-l));
    return top == -INFINITY ? 0.f : quick_exp(l - top) * inv_total;
}

// The best two keys of a lane's registers and their experts, without those whose
// bit is set in `gone`.
struct Two {
    uint32_t k1, k2;
    int e1, e2;
};
template <int NR, bool SOME_GONE>
__device__ __forceinline__ Two best_two(const uint32_t (&key)[NR], uint32_t gone, int lane)
{
    Two b{0, 0, lane, lane};
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const uint32_t v = SOME_GONE && (gone >> i & 1u) ? 0u : key[i];
        const bool first = v > b.k1, second = v > b.k2;
        b.e2 = first ? b.e1 : second ? i * 32 + lane : b.e2;
        b.k2 = max(b.k2, min(v, b.k1));
        b.e1 = first ? i * 32 + lane : b.e1;
        b.k1 = max(b.k1, v);
    }
    return b;
}

// The largest key that a warp's lanes have left, and its lowest expert.
struct Best {
    uint32_t key;
    int index;
};
__device__ __forceinline__ Best best_of(const Two &b)
{
    Best r;
    r.key = __reduce_max_sync(kAll, b.k1);
    r.index = int(__reduce_min_sync(kAll, b.k1 == r.key ? unsigned(b.e1) : 0x7fffffffu));
    return r;
}
// Takes it out.  Few lanes have three of a token's experts: only then the
// registers are read again.
template <int NR>
__device__ __forceinline__ void take(const uint32_t (&key)[NR], Two &b, uint32_t &removed, const Best &best, int lane)
{
    const bool mine = b.k1 == best.key && b.e1 == best.index;
    if (mine) {
        removed |= 1u << (best.index / 32);
        b.k1 = b.k2;
        b.e1 = b.e2;
        b.k2 = 0;
    }
    if (NR > 2 && __any_sync(kAll, mine && b.k1 == 0)) b = best_two<NR, true>(key, removed, lane);
}

// A bound of |fp32 key - exact key|, `most` being the row's largest score.  With
// u = 2^-24: exp2 is within 4 u, the rounded exponent moves it by 2 u |l|, and what
// moves exp(-l) relatively moves a sigmoid s by s (1 - s) times that: by 1.5 u in all,
// as s (1 - s) is at most 1/4 and |l| s (1 - s) below 0.23.  1 + exp(-l) and its
// reciprocal add 3 u s: below 8 u, though not below 8 u s, as exp(-l) is off by 2 u |l|
// where s is small.  In a softmax the exponent's rounding moves exp(-x), x = max - l,
// by 2 u x, which is below u in all; its sum of up to 1024 terms, 32 a lane and 5
// steps, is off by at most 37 + 4 u and 2 u times the mean of x under the softmax,
// which is below ln 1024.  The bias adds a rounding of the key.  Finite for every
// finite key.
__device__ __forceinline__ float key_error(float most, float key, bool is_sigmoid)
{
    return 0x1p-24f * (is_sigmoid ? 8.f : 1.f + 64.f * most) + 0x1p-23f * fabsf(key);
}

// Keys in 64 bits, of finite ones: all others are certain.
struct Exact {
    double top, total;  // softmax: the largest logit and the sum of exponentials
};
template <class T>
__device__ __noinline__ Exact exact_total(const T *row, int n)
{
    const int lane = int(threadIdx.x) % 32;
    double m = -INFINITY, z = 0.0;
    for (int e = lane; e < n; e += 32) m = fmax(m, double(to_f32(row[e])));
    m = warp_max(m);
    for (int e = lane; e < n; e += 32) z += exp(double(to_f32(row[e])) - m);
    return {m, warp_sum(z)};
}
__device__ __noinline__ double exact_key(float l, float b, bool is_sigmoid, Exact x)
{
    const double s = is_sigmoid          ? 1.0 / (1.0 + exp(-double(l)))
                     : x.top == -INFINITY ? 0.0
                                          : exp(double(l) - x.top) / x.total;
    return s + double(b);
}

// Which of the groups marked in `open` (bit g) come first in 64 bits: `count` of
// them, as a mask.  `bar` (in lane g): experts of group g with a lower fp32 key
// are certainly not among its best two.  Every lane lists its experts in question,
// so that the lanes form their keys side by side.
template <class T, int NR>
__device__ __noinline__ uint32_t exact_groups(const Route &p, const T *row, uint32_t open, int count, float bar, float top,
                                              float inv_total)
{
    const int lane = int(threadIdx.x) % 32, size = p.n / p.groups;
    const Exact x = p.sigmoid ? Exact{0.0, 1.0} : exact_total(row, p.n);
    int listed[NR], n = 0;  // of the experts lane, lane + 32, ..
    double key[NR];
    for (uint32_t left = open; left; left &= left - 1) {
        const int g = __ffs(int(left)) - 1;
        const float least = __shfl_sync(kAll, bar, g);
        for (int e = g * size + ((lane - g * size) & 31); e < (g + 1) * size; e += 32)
            if (quick_score(to_f32(row[e]), p.sigmoid, top, inv_total) + (p.bias ? p.bias[e] : 0.f) >= least) listed[n++] = e;
        __syncwarp();
    }
    for (int i = 0; i < n; ++i)
        key[i] = exact_key(to_f32(row[listed[i]]), p.bias ? p.bias[listed[i]] : 0.f, p.sigmoid, x);
    __syncwarp();
    double mine = -INFINITY;  // lane g: group g's score
    for (uint32_t left = open; left; left &= left - 1) {
        const int g = __ffs(int(left)) - 1;
        double k1 = -INFINITY, k2 = -INFINITY;
        for (int i = 0; i < n; ++i) {
            if (listed[i] / size != g) continue;
            k2 = fmax(k2, fmin(key[i], k1));
            k1 = fmax(k1, key[i]);
        }
        __syncwarp();
        const double first = warp_max(k1);
        double sum = first;
        if (p.group_scores == 2 && size > 1) {
            const int owner = __ffs(int(__ballot_sync(kAll, k1 == first))) - 1;
            sum += warp_max(lane == owner ? k2 : k1);
        }
        if (lane == g) mine = sum;
    }
    uint32_t chosen = 0;
    for (int r = 0; r < count; ++r) {
        const bool can = open >> lane & ~chosen >> lane & 1u;
        const double m = warp_max(can ? mine : -INFINITY);
        const unsigned at = __ballot_sync(kAll, can && mine == m);
        chosen |= at & (0u - at);
    }
    return chosen;
}

// The choices from the `from`-th on again, in 64 bits, among the experts marked in
// `open` (bit i: expert i * 32 + lane): all that can be among them.  Lane j: the
// j-th.
template <class T, int NR>
__device__ __noinline__ int exact_choice(const Route &p, const T *row, uint32_t open, int from)
{
    const int lane = int(threadIdx.x) % 32;
    const Exact x = p.sigmoid ? Exact{0.0, 1.0} : exact_total(row, p.n);
    double key[NR];
    for (uint32_t left = open; left; left &= left - 1) {
        const int i = __ffs(int(left)) - 1, e = i * 32 + lane;
        key[i] = exact_key(to_f32(row[e]), p.bias[e], p.sigmoid, x);
    }
    __syncwarp();
    int chosen = 0;
    for (int j = from; j < p.top; ++j) {
        double k = -INFINITY;
        int at = -1;
        for (uint32_t left = open; left; left &= left - 1) {
            const int i = __ffs(int(left)) - 1;
            if (at < 0 || key[i] > k) {
                k = key[i];
                at = i;
            }
        }
        __syncwarp();
        const double m = warp_max(k);
        const int index = int(__reduce_min_sync(kAll, at >= 0 && k == m ? unsigned(at * 32 + lane) : 0x7fffffffu));
        if (at >= 0 && index == at * 32 + lane) open &= ~(1u << at);
        if (lane == j) chosen = index;
    }
    return chosen;
}

// The chosen experts (lane j: the j-th) put in order again: lane j and the next
// one change places while both are marked in `doubtful` and their keys in 64 bits
// stand the other way round.  All others' order is certain.
template <class T>
__device__ __noinline__ int exact_order(const Route &p, const T *row, int index, unsigned doubtful)
{
    const int lane = int(threadIdx.x) % 32;
    const Exact x = p.sigmoid ? Exact{0.0, 1.0} : exact_total(row, p.n);
    const bool mine = doubtful >> lane & 1u;
    double key = mine ? exact_key(to_f32(row[index]), p.bias[index], p.sigmoid, x) : 0.0;
    __syncwarp();
    for (int r = 0; r < p.top; ++r) {  // neighbours (0, 1), (2, 3) .., then (1, 2), (3, 4) ..
        const int other = (lane + r) % 2 == 0 ? lane + 1 : lane - 1;
        const double k = __shfl_sync(kAll, key, other & 31);
        const int i = __shfl_sync(kAll, index, other & 31);
        if (mine && other >= 0 && other < 32 && (doubtful >> other & 1u)) {
            const bool first = key > k || (key == k && index < i);  // this one belongs before the other
            if (first != (lane < other)) {
                key = k;
                index = i;
            }
        }
    }
    return index;
}

template <class T, int NR, bool FULL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const Route p)
{
    const int lane = int(threadIdx.x) % 32;
    const int64_t t = int64_t(blockIdx.x) * kRouteWarps + threadIdx.x / 32;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.tokens) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ld;
    float l[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) l[i] = FULL || i * 32 + lane < p.n ? to_f32(row[i * 32 + lane]) : 0.f;
    uint32_t closed = 0;  // bit i: expert i * 32 + lane cannot be chosen (any more)
#pragma unroll
    for (int i = 0; i < NR; ++i) closed |= FULL || i * 32 + lane < p.n ? 0u : 1u << i;

    // softmax over all experts, where the weights or the keys need it
    float top = 0.f, total = 1.f, inv_total = 1.f;
    if (!p.sigmoid && (!p.renorm || p.bias || p.score_groups)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) m = max(m, closed >> i & 1u ? 0u : ordered(l[i]));
        m = __reduce_max_sync(kAll, m);
        top = unordered(m);
        total = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) total += closed >> i & 1u || top == -INFINITY ? 0.f : expf(l[i] - top);
        total = warp_sum(total);
        inv_total = top == -INFINITY ? 0.f : 1.f / total;
    }
    // a row whose logits are all -inf has no scores, and its keys no error but the bias's
    auto score = [&](float v) {
        return p.sigmoid ? sigmoid(v) : top == -INFINITY ? 0.f : expf(v - top) / total;
    };
    const float most_score = p.sigmoid ? 1.f : inv_total;  // no score of the row is larger
    uint32_t key[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int e = i * 32 + lane;
        float k = l[i];
        if (p.bias || p.score_groups) k = quick_score(k, p.sigmoid, top, inv_total);
        if (p.bias && (FULL || e < p.n)) k += p.bias[e];
        key[i] = FULL || e < p.n ? ordered(k) : 0u;
    }

    if (p.top_groups < p.groups) {
        const int size = p.n / p.groups;
        uint32_t most1 = 0, most2 = 0;  // lane g: group g's best two keys
        auto close_group = [&](int g, uint32_t k1, uint32_t k2) {
            const uint32_t m = __reduce_max_sync(kAll, k1);
            const unsigned at = __ballot_sync(kAll, k1 == m);
            const uint32_t second = __reduce_max_sync(kAll, at & (0u - at) & 1u << lane ? k2 : k1);
            if (lane == g) {
                most1 = m;
                most2 = second;
            }
        };
        if (size % 32 == 0) {  // whole registers
            uint32_t k1 = 0, k2 = 0;
            int g = 0, until = size / 32;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                k2 = max(k2, min(key[i], k1));
                k1 = max(k1, key[i]);
                if (i + 1 == until && g < p.groups) {
                    close_group(g++, k1, k2);
                    until += size / 32;
                    k1 = k2 = 0;
                }
            }
        } else {
            for (int g = 0; g < p.groups; ++g) {
                const int first = g * size, last = first + size - 1;
                uint32_t k1 = 0, k2 = 0;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    if (i < first / 32 || i > last / 32) continue;
                    const int e = i * 32 + lane;
                    const uint32_t v = e >= first && e <= last ? key[i] : 0u;
                    k2 = max(k2, min(v, k1));
                    k1 = max(k1, v);
                }
                close_group(g, k1, k2);
            }
        }
        uint32_t mine = most1;  // lane g: group g's score, of two keys half of it: the sum of two large biases is infinite
        float error = 0.f, bar = 0.f;  // where the score is finite: infinite ones and NaN are certain
        if (lane < p.groups) {
            const float a = unordered(most1);
            float least = a;
            if (p.bias || p.score_groups) error = key_error(most_score, a, p.sigmoid);
            if (p.group_scores == 2 && size > 1) {
                const float b = unordered(most2), half = 0.5f * a + 0.5f * b;
                mine = ordered(half);
                error = 0.5f * error + 0.5f * key_error(most_score, b, p.sigmoid) + 0x1p-23f * fabsf(half);
                least = b;
            }
            bar = least - 2.f * (p.bias || p.score_groups ? key_error(most_score, least, p.sigmoid) : 0.f);
        }
        int before = 0;  // groups that come before this lane's
        for (int g = 0; g < p.groups; ++g) {
            const uint32_t v = __shfl_sync(kAll, mine, g);
            before += v > mine || (v == mine && g < lane);
        }
        const bool kept = lane < p.groups && before < p.top_groups;
        uint32_t chosen = __ballot_sync(kAll, kept);
        if (p.bias || p.score_groups) {
            // In doubt is a kept group that may lie below what one that is not kept may reach,
            // and the other way round.  Each has its own error: that of a group with a bias of
            // 1e30 does not make the others near.
            const float score = unordered(mine);
            const bool here = lane < p.groups && is_finite(score);
            const uint32_t low = ordered(score - error), high = ordered(score + error);
            const uint32_t least = __reduce_min_sync(kAll, here && kept ? low : kNan), most = __reduce_max_sync(kAll, here && !kept ? high : 0u);
            if (least <= most) {
                const uint32_t open = __ballot_sync(kAll, here && (kept ? low <= most : high >= least)), sure = chosen & ~open;
                chosen = sure | exact_groups<T, NR>(p, row, open, p.top_groups - __popc(sure), bar, top, inv_total);
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int e = i * 32 + lane;
            if ((FULL || e < p.n) && !(chosen >> (unsigned(e) * p.inv_size >> 20) & 1u)) {
                closed |= 1u << i;
                if (p.bias || !p.score_groups) key[i] = 0u;
            }
        }
    }

    if (!p.bias && p.score_groups) {  // among the open experts scores have the order of logits
#pragma unroll
        for (int i = 0; i < NR; ++i) key[i] = closed >> i & 1u ? 0u : ordered(l[i]);
    }
    int index = 0;  // lane j: the j-th expert
    uint32_t mine = 0, removed = closed, next = 0;
    int next_index = -1;
    Two two = best_two<NR, false>(key, 0u, lane);  // closed ones are 0
    for (int j = 0; j < p.top; ++j) {
        const Best b = best_of(two);
        take<NR>(key, two, removed, b, lane);
        if (lane == j) {
            index = b.index;
            mine = b.key;
        }
    }
    float logit = lane < p.top ? to_f32(row[index]) : 0.f;
    if (p.bias) {
        const Best b = best_of(two);  // the first that was not chosen
        next = b.key;
        next_index = b.key ? b.index : -1;
        // Each chosen key against the next one.  Equal logits and biases are equal keys,
        // whose order is that of the indices; others that near are ordered in 64 bits,
        // together with all that are as near or equal to them.
        const float bias = lane < p.top ? p.bias[index] : 0.f;
        float l1 = __shfl_down_sync(kAll, logit, 1), b1 = __shfl_down_sync(kAll, bias, 1);
        uint32_t k1 = __shfl_down_sync(kAll, mine, 1);
        if (lane == p.top - 1) {
            k1 = next;
            l1 = next_index >= 0 ? to_f32(row[next_index]) : 0.f;
            b1 = next_index >= 0 ? p.bias[next_index] : 0.f;
        }
        const float ka = unordered(mine), kb = unordered(k1);
        // Infinite keys and NaN come from a bias (or a logit) alone, without an error: their order is certain.
        const bool both = lane < p.top && k1 != 0u && is_finite(ka) && is_finite(kb), equal = l1 == logit && b1 == bias;
        // the errors are those of the row's largest score: what is not near to its neighbour is not near to any further one
        const bool close = both && (equal || ka - kb <= key_error(most_score, ka, p.sigmoid) + key_error(most_score, kb, p.sigmoid));
        const unsigned linked = __ballot_sync(kAll, close);
        unsigned near = __ballot_sync(kAll, close && !equal);
        bool border = linked >> (p.top - 1) & 1u;
        const float last = __shfl_sync(kAll, ka, p.top - 1);
        // what lies further below the last chosen key than both errors, of the row's largest score, is not among the best
        const uint32_t least = ordered(last - 2.f * key_error(most_score, last, p.sigmoid));
        if (border && !near) {  // equal to the last one: is any other as near?
            const float ll = __shfl_sync(kAll, logit, p.top - 1), bl = __shfl_sync(kAll, bias, p.top - 1);
            bool other = false;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int e = i * 32 + lane;
                if (!(removed >> i & 1u) && key[i] >= least) other |= to_f32(row[e]) != ll || p.bias[e] != bl;
            }
            near = __any_sync(kAll, other);
        }
        if (near) {
            unsigned doubtful = linked | linked << 1;
            if (border) {  // who is chosen is in doubt, from the first choice on that is linked to the last
                const unsigned others = ~linked & ((1u << (p.top - 1)) - 1u);
                const int from = others ? 32 - __clz(int(others)) : 0;
                const uint32_t largest = __shfl_sync(kAll, mine, from);
                uint32_t open = 0;
#pragma unroll
                for (int i = 0; i < NR; ++i) open |= key[i] >= least && key[i] <= largest ? 1u << i : 0u;
                const int again = exact_choice<T, NR>(p, row, open, from);
                if (lane >= from && again < p.n) index = again;
                doubtful = (linked & ((1u << from) - 1u)) | (linked & ((1u << from) - 1u)) << 1;
                doubtful &= (1u << from) - 1u;
            }
            if (doubtful) index = exact_order<T>(p, row, index, doubtful);
        }
        if (near && lane < p.top) logit = to_f32(row[index]);
    }

    float w = 0.f;
    const bool have = lane < p.top;
    if (p.renorm) {
        // scores relative to the largest chosen one's scale, so that none vanishes before the quotient
        uint32_t m = have ? ordered(logit) : 0u;
        m = __reduce_max_sync(kAll, m);
        const float largest = unordered(m);
        const float shift = p.sigmoid ? fminf(largest, 0.f) : largest;
        float v = 0.f;
        if (have && largest != -INFINITY) {
            v = p.sigmoid ? relative_sigmoid(logit, shift) : expf(logit - shift);
        }
        if (m == kNan || total != total) v = NAN;  // total: a softmax that met one elsewhere in the row
        const float sum = warp_sum(have ? v : 0.f);
        w = sum == 0.f ? 0.f : v / sum * p.scale;
    } else if (have) {
        w = score(logit) * p.scale;
    }
    if (have) {
        p.weights[t * p.top + lane] = w;
        p.experts[t * p.top + lane] = index;
    }
}

struct RouteBackward {
    const float *dweights;
    const void *logits;
    int64_t ld, tokens;
    const int *experts;
    void *dlogits;
    int n, top;
    bool sigmoid, renorm;
    float scale;
};

// One warp a token again.  With p_j = s_j (renormalised: s_j / sum of the chosen)
// and q = sum_i p_i dw_i over the chosen:
//   renormalised   softmax: dl_j = scale p_j (dw_j - q),  sigmoid: times 1 - s_j
//   as they are    softmax: dl_e = scale p_e ([e chosen] dw_e - q) for every e,
//                  sigmoid: dl_j = scale dw_j s_j (1 - s_j)
// Lane j forms what belongs to the j-th choice.  The row is written as it is for
// experts that were not chosen, and then the chosen ones' elements over it; an
// expert given twice gets both parts, from the first of its lanes.
template <class T, int NR>
__global__ void __launch_bounds__(32 * kRouteWarps) route_backward_kernel(const RouteBackward p)
{
    const int lane = int(threadIdx.x) % 32;
    const int64_t t = int64_t(blockIdx.x) * kRouteWarps + threadIdx.x / 32;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.tokens) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ld;
    T *out = static_cast<T *>(p.dlogits) + t * p.n;
    int index = -1;
    float dw = 0.f, logit = 0.f;
    if (lane < p.top) {
        index = p.experts[t * p.top + lane];
        dw = p.dweights[t * p.top + lane];
        if (index < 0 || index >= p.n) index = -1;  // not routed: takes no part
    }
    const bool have = index >= 0;
    float part = 0.f, rest = 0.f;  // of the chosen expert alone; what it has in common with all others
    if (!p.sigmoid && !p.renorm) {
        float l[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) l[i] = i * 32 + lane < p.n ? to_f32(row[i * 32 + lane]) : -INFINITY;
        if (have) logit = to_f32(row[index]);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) m = max(m, i * 32 + lane < p.n ? ordered(l[i]) : 0u);
        m = __reduce_max_sync(kAll, m);
        const float top = unordered(m);
        float total = 0.f, dl[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            dl[i] = top == -INFINITY || i * 32 + lane >= p.n ? 0.f : expf(l[i] - top);
            total += dl[i];
        }
        total = warp_sum(total);
        const float inv = total == 0.f ? 0.f : 1.f / total;
        const float s = have && top != -INFINITY ? expf(logit - top) * inv : 0.f;
        const float q = warp_sum(have ? s * dw : 0.f);
        part = s * dw * p.scale;
        rest = -s * q * p.scale;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (i * 32 + lane < p.n) out[i * 32 + lane] = from_f32<T>(dl[i] * (-inv * q * p.scale));
    } else {
        if (have) logit = to_f32(row[index]);
        if (!p.renorm) {
            const float s = sigmoid(logit);
            part = have ? p.scale * dw * s * sigmoid(-logit) : 0.f;
        } else {
            uint32_t m = __reduce_max_sync(kAll, have ? ordered(logit) : 0u);
            const float largest = m == 0u ? -INFINITY : unordered(m);
            const float shift = p.sigmoid ? fminf(largest, 0.f) : largest;
            float v = 0.f;
            if (have && largest != -INFINITY) {
                v = p.sigmoid ? relative_sigmoid(logit, shift) : expf(logit - shift);
            }
            if (m == kNan) v = have ? NAN : 0.f;
            const float sum = warp_sum(v);
            const float share = sum == 0.f ? 0.f : v / sum;
            const float q = warp_sum(have ? share * dw : 0.f);
            part = have ? p.scale * share * (dw - q) * (p.sigmoid ? sigmoid(-logit) : 1.f) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (i * 32 + lane < p.n) out[i * 32 + lane] = from_f32<T>(0.f);
    }
    __syncwarp();  // the row's elements are written before those of the chosen experts
    float sum = 0.f;
    bool first = have;
    for (int j = 0; j < p.top; ++j) {
        const int e = __shfl_sync(kAll, index, j);
        const float v = __shfl_sync(kAll, part, j);
        if (e == index) {
            sum += v;
            if (j < lane) first = false;
        }
    }
    if (first) out[index] = from_f32<T>(sum + rest);
}

// Calls f with the smallest of 1, 2, 4 .. 32 registers that hold `n` experts.
template <class F>
static int with_registers(int n, F f)
{
    if (n <= 32) return f(std::integral_constant<int, 1>{});
    if (n <= 64) return f(std::integral_constant<int, 2>{});
    if (n <= 128) return f(std::integral_constant<int, 4>{});
    if (n <= 256) return f(std::integral_constant<int, 8>{});
    if (n <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

template <class T>
static int route(const Route &p, cudaStream_t s)
{
    const dim3 grid(unsigned((p.tokens + kRouteWarps - 1) / kRouteWarps));
    return with_registers(p.n, [&](auto nr) {
        constexpr int NR = decltype(nr)::value;
        return p.n == NR * 32 ? launch(route_kernel<T, NR, true>, grid, dim3(32 * kRouteWarps), 0, s, 1, p)
                              : launch(route_kernel<T, NR, false>, grid, dim3(32 * kRouteWarps), 0, s, 1, p);
    });
}

template <class T>
static int route_backward(const RouteBackward &p, cudaStream_t s)
{
    const dim3 grid(unsigned((p.tokens + kRouteWarps - 1) / kRouteWarps));
    return with_registers(p.n, [&](auto nr) {
        return launch(route_backward_kernel<T, decltype(nr)::value>, grid, dim3(32 * kRouteWarps), 0, s, 1, p);
    });
}

// What both directions ask of their sizes, and a GB300.
static int check_route(int64_t tokens, int64_t experts, int top, int dtype, int scoring)
{
    if (dtype != kF16 && dtype != kBF16 && dtype != kF32) return kErrUnsupportedDtype;
    if (tokens < 0 || tokens > 2147483647 || experts < 1 || experts > kMaxExperts || top < 1 || top > kMaxTop || top > experts)
        return kErrInvalidArg;
    if (scoring != TGEMM_SOFTMAX && scoring != TGEMM_SIGMOID) return kErrInvalidArg;
    return kOk;
}

static int check_gb300()
{
    Device d;
    const int rc = current_device(d);
    if (rc != kOk) return rc;
    return d.gb300 ? kOk : kErrArch;
}

static bool off(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % unsigned(bytes) != 0; }

}  // namespace tg

using namespace tg;

extern "C" {

int tgemm_route(int64_t tokens, int64_t experts, int top, int dtype, const void *logits, int64_t ld, const float *bias,
                int scoring, int groups, int top_groups, int group_scores, int renormalize, float scale, float *weights,
                int *chosen, tgemm_stream_t stream)
{
    int rc = check_route(tokens, experts, top, dtype, scoring);
    if (rc != kOk) return rc;
    if (groups < 1 || groups > kMaxGroups || experts % groups || top_groups < 1 || top_groups > groups || group_scores < 1 ||
        group_scores > 2 || top > experts / groups * top_groups)
        return kErrInvalidArg;
    if ((rc = check_gb300()) != kOk) return rc;
    if (tokens == 0) return kOk;
    if (!logits || !weights || !chosen || ld < experts) return kErrInvalidArg;
    if (off(logits, dtype_bytes(dtype)) || off(bias, 4) || off(weights, 4) || off(chosen, 4)) return kErrAlignment;
    Route p{};
    p.logits = logits;
    p.ld = ld;
    p.tokens = tokens;
    p.bias = bias;
    p.weights = weights;
    p.experts = chosen;
    p.n = int(experts);
    p.top = top;
    p.groups = groups;
    p.top_groups = top_groups;
    p.group_scores = group_scores;
    p.sigmoid = scoring == TGEMM_SIGMOID;
    p.renorm = renormalize != 0;
    p.inv_size = unsigned(((1 << 20) + experts / groups - 1) / (experts / groups));
    p.score_groups = top_groups < groups && group_scores == 2;
    p.scale = scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == kF32 ? route<float>(p, s) : dtype == kF16 ? route<__half>(p, s) : route<__nv_bfloat16>(p, s);
}

int tgemm_route_backward(int64_t tokens, int64_t experts, int top, int dtype, const float *dweights, const void *logits,
                         int64_t ld, const int *chosen, int scoring, int renormalize, float scale, void *dlogits,
                         tgemm_stream_t stream)
{
    int rc = check_route(tokens, experts, top, dtype, scoring);
    if (rc != kOk) return rc;
    if ((rc = check_gb300()) != kOk) return rc;
    if (tokens == 0) return kOk;
    if (!dweights || !logits || !chosen || !dlogits || ld < experts) return kErrInvalidArg;
    const int e = dtype_bytes(dtype);
    if (off(logits, e) || off(dlogits, e) || off(dweights, 4) || off(chosen, 4)) return kErrAlignment;
    RouteBackward p{};
    p.dweights = dweights;
    p.logits = logits;
    p.ld = ld;
    p.tokens = tokens;
    p.experts = chosen;
    p.dlogits = dlogits;
    p.n = int(experts);
    p.top = top;
    p.sigmoid = scoring == TGEMM_SIGMOID;
    p.renorm = renormalize != 0;
    p.scale = scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == kF32   ? route_backward<float>(p, s)
           : dtype == kF16 ? route_backward<__half>(p, s)
                           : route_backward<__nv_bfloat16>(p, s);
}

}  // extern "C"
