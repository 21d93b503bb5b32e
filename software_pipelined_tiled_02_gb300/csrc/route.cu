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
// again in 64 bits: about one token in a thousand.
//
// What bounds it: at 8192 tokens and 256 experts 8.9 MB move in 1.3 us; the
// rounds' instructions and, for the few tokens with near ties, the 64-bit
// exponentials take longer.

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"
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
    bool score_groups;  // the groups' scores come from scores, not from logits
    float scale;
};

// fp32 values as unsigned integers of the same order: -0 as +0, every NaN above
// all others, nothing below 1 (0 stands for "no value").
__device__ __forceinline__ uint32_t ordered(float v)
{
    if (v != v) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

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

// The largest key that a warp's lanes have left, and its lowest index.
struct Best {
    uint32_t key;
    int index;
};
template <int NR>
__device__ __forceinline__ Best best_of(const uint32_t (&key)[NR], uint32_t removed, int lane)
{
    uint32_t k = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const uint32_t v = removed >> i & 1u ? 0u : key[i];
        if (v > k) {
            k = v;
            at = i;
        }
    }
    Best b;
    b.key = __reduce_max_sync(kAll, k);
    b.index = int(__reduce_min_sync(kAll, k == b.key && k ? unsigned(at * 32 + lane) : 0x7fffffffu));
    return b;
}

// A bound of |fp32 key - exact key|.  With u = 2^-24: expf is within 2 ulp (4 u),
// the sum and the quotient add a rounding each, so a sigmoid is within 6 u s.  In
// a softmax the rounded difference x = max - l moves exp(-x) by another u x, which
// is at most 0.4 u in all; the sum of up to 1024 terms, 32 a lane and 5 steps, is
// off by at most 37 + 4 u and u times the mean of x under the softmax, which is
// below ln 1024.  The bias adds a rounding of the key.
__device__ __forceinline__ float key_error(float s, float key) { return 0x1p-24f * (1.f + 64.f * s + 2.f * fabsf(key)); }

// Keys in 64 bits.
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

// The groups' choice again in 64 bits: bit g of the result is group g.
template <class T>
__device__ __noinline__ uint32_t exact_groups(const Route &p, const T *row)
{
    const int lane = int(threadIdx.x) % 32, size = p.n / p.groups;
    const Exact x = p.sigmoid ? Exact{0.0, 1.0} : exact_total(row, p.n);
    double mine = -INFINITY;  // lane g: group g's score
    for (int g = 0; g < p.groups; ++g) {
        double k1 = -INFINITY, k2 = -INFINITY;
        for (int e = g * size + lane; e < (g + 1) * size; e += 32) {
            const double k = exact_key(to_f32(row[e]), p.bias ? p.bias[e] : 0.f, p.sigmoid, x);
            k2 = fmax(k2, fmin(k, k1));
            k1 = fmax(k1, k);
        }
        const double first = warp_max(k1);
        if (p.group_scores == 2 && size > 1) {
            const int owner = __ffs(int(__ballot_sync(kAll, k1 == first))) - 1;
            const double second = warp_max(lane == owner ? k2 : k1);
            if (lane == g) mine = first + second;
        } else if (lane == g) {
            mine = first;
        }
    }
    uint32_t chosen = 0;
    for (int r = 0; r < p.top_groups; ++r) {
        const bool open = lane < p.groups && !(chosen >> lane & 1u);
        const double m = warp_max(open ? mine : -INFINITY);
        const unsigned at = __ballot_sync(kAll, open && mine == m);
        chosen |= at & (0u - at);
    }
    return chosen;
}

// The choice of experts again, in 64 bits, among those marked in `open` (bit i:
// expert i * 32 + lane), every expert that can be among the best.
template <class T, int NR>
__device__ __noinline__ int exact_choice(const Route &p, const T *row, uint32_t open)
{
    const int lane = int(threadIdx.x) % 32;
    const Exact x = p.sigmoid ? Exact{0.0, 1.0} : exact_total(row, p.n);
    double key[NR];
    for (int i = 0; i < NR; ++i) {
        const int e = i * 32 + lane;
        key[i] = 0.0;
        if (open >> i & 1u) {
            const double k = exact_key(to_f32(row[e]), p.bias[e], p.sigmoid, x);
            key[i] = k != k ? double(INFINITY) : fmin(k, 1e300);  // NaN above all others
        }
    }
    int chosen = 0;
    for (int j = 0; j < p.top; ++j) {
        double k = -INFINITY;
        int at = -1;
        for (int i = 0; i < NR; ++i) {
            if ((open >> i & 1u) && (at < 0 || key[i] > k)) {
                k = key[i];
                at = i;
            }
        }
        const double m = warp_max(k);
        const int index = int(__reduce_min_sync(kAll, at >= 0 && k == m ? unsigned(at * 32 + lane) : 0x7fffffffu));
        if (at >= 0 && index == at * 32 + lane) open &= ~(1u << at);
        if (lane == j) chosen = index;
    }
    return chosen;
}

template <class T, int NR>
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
    for (int i = 0; i < NR; ++i) l[i] = i * 32 + lane < p.n ? to_f32(row[i * 32 + lane]) : 0.f;
    uint32_t closed = 0;  // bit i: expert i * 32 + lane cannot be chosen (any more)
#pragma unroll
    for (int i = 0; i < NR; ++i) closed |= i * 32 + lane < p.n ? 0u : 1u << i;

    // softmax over all experts, where the weights or the keys need it
    float top = 0.f, total = 1.f;
    if (!p.sigmoid && (!p.renorm || p.bias || p.score_groups)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) m = max(m, closed >> i & 1u ? 0u : ordered(l[i]));
        m = __reduce_max_sync(kAll, m);
        top = m == 0xffffffffu ? NAN : unordered(m);
        total = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) total += closed >> i & 1u || top == -INFINITY ? 0.f : expf(l[i] - top);
        total = warp_sum(total);
    }
    // a row whose logits are all -inf has no scores
    auto score = [&](float v) {
        return p.sigmoid ? sigmoid(v) : top == -INFINITY ? 0.f : expf(v - top) / total;
    };
    uint32_t key[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int e = i * 32 + lane;
        key[i] = ordered(!p.bias && !p.score_groups ? l[i] : score(l[i]) + (p.bias && e < p.n ? p.bias[e] : 0.f));
    }

    if (p.top_groups < p.groups) {
        const int size = p.n / p.groups;
        uint32_t mine = 0;  // lane g: group g's score
        float error = 0.f;
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
            uint32_t m = __reduce_max_sync(kAll, k1);
            float err = 0.f;
            if (p.group_scores == 2 && size > 1) {
                const int owner = __ffs(int(__ballot_sync(kAll, k1 == m))) - 1;
                const uint32_t second = __reduce_max_sync(kAll, lane == owner ? k2 : k1);
                const float a = m == 0xffffffffu ? NAN : unordered(m), b = second == 0xffffffffu ? NAN : unordered(second);
                m = ordered(a + b);
                err = key_error(1.f, a) + key_error(1.f, b) + 0x1p-24f * fabsf(a + b);
            } else if (p.bias || p.score_groups) {
                err = key_error(1.f, m == 0xffffffffu ? 0.f : unordered(m));
            }
            if (lane == g) {
                mine = m;
                error = err;
            }
        }
        uint32_t chosen = 0, last = 0;
        float last_error = 0.f;
        for (int r = 0; r <= p.top_groups; ++r) {
            const uint32_t v = lane < p.groups && !(chosen >> lane & 1u) ? mine : 0u;
            const uint32_t m = __reduce_max_sync(kAll, v);
            const unsigned at = __ballot_sync(kAll, v == m && lane < p.groups && !(chosen >> lane & 1u));
            const float e = __shfl_sync(kAll, error, __ffs(int(at)) - 1);
            if (r < p.top_groups) {
                chosen |= at & (0u - at);
                last = m;
                last_error = e;
            } else if (last != 0xffffffffu && unordered(last) - unordered(m) <= e + last_error && e + last_error > 0.f) {
                chosen = exact_groups<T>(p, row);
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int e = i * 32 + lane;
            if (e < p.n && !(chosen >> (e / size) & 1u)) closed |= 1u << i;
        }
    }

    if (!p.bias && p.score_groups) {  // among the open experts scores have the order of logits
#pragma unroll
        for (int i = 0; i < NR; ++i) key[i] = ordered(l[i]);
    }
    int index = 0;  // lane j: the j-th expert
    uint32_t mine = 0, removed = closed, next = 0;
    int next_index = -1;
    for (int j = 0; j < p.top; ++j) {
        const Best b = best_of<NR>(key, removed, lane);
        if (b.index % 32 == lane) removed |= 1u << (b.index / 32);
        if (lane == j) {
            index = b.index;
            mine = b.key;
        }
    }
    float logit = lane < p.top ? to_f32(row[index]) : 0.f;
    if (p.bias) {
        const Best b = best_of<NR>(key, removed, lane);  // the first that was not chosen
        next = b.key;
        next_index = b.key ? b.index : -1;
        // Each chosen key against the next one: equal logits and biases are equal
        // keys; others that near are ordered in 64 bits.
        const float bias = lane < p.top ? p.bias[index] : 0.f;
        float l1 = __shfl_down_sync(kAll, logit, 1), b1 = __shfl_down_sync(kAll, bias, 1);
        uint32_t k1 = __shfl_down_sync(kAll, mine, 1);
        if (lane == p.top - 1) {
            k1 = next;
            l1 = next_index >= 0 ? to_f32(row[next_index]) : 0.f;
            b1 = next_index >= 0 ? p.bias[next_index] : 0.f;
        }
        const bool both = lane < p.top && k1 != 0u && mine != 0xffffffffu && (l1 != logit || b1 != bias);
        const float ka = unordered(mine), kb = unordered(k1);
        const bool near = both && ka - kb <= key_error(score(logit), ka) + key_error(score(l1), kb);
        if (__any_sync(kAll, near)) {
            const float last = __shfl_sync(kAll, ka, p.top - 1);
            // what lies further below the last chosen key than both errors, of scores up to 1, is not among the best
            const uint32_t bar = ordered(last - 2.f * key_error(1.f, last));
            uint32_t open = 0;
#pragma unroll
            for (int i = 0; i < NR; ++i) open |= !(closed >> i & 1u) && key[i] >= bar ? 1u << i : 0u;
            index = exact_choice<T, NR>(p, row, open);
            if (lane < p.top) logit = to_f32(row[index]);
        }
    }

    float w = 0.f;
    const bool have = lane < p.top;
    if (p.renorm) {
        // scores relative to the largest chosen one's scale, so that none vanishes before the quotient
        uint32_t m = have ? ordered(logit) : 0u;
        m = __reduce_max_sync(kAll, m);
        const float largest = m == 0xffffffffu ? NAN : unordered(m);
        const float shift = p.sigmoid ? fminf(largest, 0.f) : largest;
        float v = 0.f;
        if (have && largest != -INFINITY) {
            if (!p.sigmoid)
                v = expf(logit - shift);
            else
                v = logit > 0.f ? sigmoid(logit) : expf(logit - shift) / (1.f + expf(logit));
        }
        if (m == 0xffffffffu || total != total) v = NAN;  // total: a softmax that met one elsewhere in the row
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
// Lane j forms what belongs to the j-th choice, and every lane picks up what
// falls to its experts, so an expert given twice gets both parts.
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
    float part = 0.f, dl[NR];
    if (!p.sigmoid && !p.renorm) {
        float l[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) l[i] = i * 32 + lane < p.n ? to_f32(row[i * 32 + lane]) : -INFINITY;
        if (have) logit = to_f32(row[index]);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) m = max(m, i * 32 + lane < p.n ? ordered(l[i]) : 0u);
        m = __reduce_max_sync(kAll, m);
        const float top = m == 0xffffffffu ? NAN : unordered(m);
        float total = 0.f;
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
#pragma unroll
        for (int i = 0; i < NR; ++i) dl[i] *= -inv * q * p.scale;
    } else {
        if (have) logit = to_f32(row[index]);
        if (!p.renorm) {
            const float s = sigmoid(logit);
            part = have ? p.scale * dw * s * sigmoid(-logit) : 0.f;
        } else {
            uint32_t m = __reduce_max_sync(kAll, have ? ordered(logit) : 0u);
            const float largest = m == 0u ? -INFINITY : m == 0xffffffffu ? NAN : unordered(m);
            const float shift = p.sigmoid ? fminf(largest, 0.f) : largest;
            float v = 0.f;
            if (have && largest != -INFINITY) {
                if (!p.sigmoid)
                    v = expf(logit - shift);
                else
                    v = logit > 0.f ? sigmoid(logit) : expf(logit - shift) / (1.f + expf(logit));
            }
            if (m == 0xffffffffu) v = have ? NAN : 0.f;
            const float sum = warp_sum(v);
            const float share = sum == 0.f ? 0.f : v / sum;
            const float q = warp_sum(have ? share * dw : 0.f);
            part = have ? p.scale * share * (dw - q) * (p.sigmoid ? sigmoid(-logit) : 1.f) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) dl[i] = 0.f;
    }
    for (int j = 0; j < p.top; ++j) {
        const int e = __shfl_sync(kAll, index, j);
        const float v = __shfl_sync(kAll, part, j);
        if (e % 32 == lane) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (i == e / 32) dl[i] += v;
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
        if (i * 32 + lane < p.n) out[i * 32 + lane] = from_f32<T>(dl[i]);
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
        return launch(route_kernel<T, decltype(nr)::value>, grid, dim3(32 * kRouteWarps), 0, s, 1, p);
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
