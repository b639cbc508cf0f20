// route.hip -- a router's selection from logits to gate weights, and the gradient
// of its logits.
//
//   p = softmax(x) | sigmoid(x);  s = p + bias;  the best groups by the sum of
//   their one or two best s;  the k best s of those;  w = scale p / (sum p | 1)
//
// Which experts are chosen has to be right to the last: s of two experts may be as
// near as the inputs make them, so s is in 64 bits (2^-52 against the 2^-24 by
// which 32 bits would swap neighbours among millions of pairs).  Where no bias and
// no sum of two scores is asked for, s orders the experts as x does, and x itself
// is compared.
//
// A token belongs to L lanes (16, so that four tokens share a wave's instructions,
// or 64), and each group of experts to a power of two of them, V neighbouring
// experts to a lane: the group's best are then found by a butterfly of a few lanes,
// and the lower index is the lower lane and the lower place in it.  The k best are
// taken one after the other, each by the largest of a lane's V and a butterfly.
#include <cmath>
#include <type_traits>

#include "ops_common.h"

namespace segtopk_ops {
namespace {

constexpr int kMaxK = 64, kMaxExperts = 1024, kMaxGroups = 64;

struct RouteArgs {
    int64_t stride;
    const float *bias;
    float *weights;
    int32_t *experts;
    uint32_t tokens, num_experts, k, groups, per_group, group_lanes, kept, best;
    uint32_t sigmoid, renormalize;
    double scale;
};

template <class X> __device__ inline X larger(X a, X b) { return a > b ? a : b; }
__device__ inline uint32_t lower(uint32_t a, uint32_t b) { return a < b ? a : b; }

// The two best of a group, kept through a butterfly.
template <class X> struct Best {
    X first, second;
};
template <int D, class X> __device__ inline void join_best(Best<X> &b) {
    const X f = partner<D>(b.first), s = partner<D>(b.second);
    b.second = larger(larger(b.second, s), b.first < f ? b.first : f);
    b.first = larger(b.first, f);
}

// log sigmoid(x), without loss where sigmoid underflows.
__device__ inline double log_sigmoid(double x) {
    return (x < 0.0 ? x : 0.0) - log1p(exp(-fabs(x)));
}

// S: the type that scores are compared in; float: they are the logits.
template <class T, class S, int L, int V>
__global__ __launch_bounds__(kOpThreads) void route_kernel(const T *logits, RouteArgs a) {
    constexpr bool kWide = sizeof(S) == 8;
    constexpr int kTokens = kOpThreads / L;
    constexpr S kNone = (S)-INFINITY;
    __shared__ float chosen_x[kTokens][kMaxK];
    __shared__ int32_t chosen[kTokens][kMaxK];
    const uint32_t lane = threadIdx.x % L, local = threadIdx.x / L;
    const uint32_t token = blockIdx.x * kTokens + local;
    // All lanes of a wave stay for the butterflies; lanes without a token have none to choose from.
    const bool live = token < a.tokens;
    const uint32_t group = lane / a.group_lanes, in_group = (lane % a.group_lanes) * V;
    const uint32_t first = group * a.per_group + in_group;
    const uint32_t mine = !live || group >= a.groups || in_group >= a.per_group
                              ? 0u
                              : (a.per_group - in_group < (uint32_t)V ? a.per_group - in_group : (uint32_t)V);
    float x[V];
    {
        typedef T mem __attribute__((ext_vector_type(V), aligned(sizeof(T))));
        const T *row = logits + (int64_t)(live ? token : 0) * a.stride + first;
        if (mine == (uint32_t)V) {
            const mem v = *reinterpret_cast<const mem *>(row);
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = (float)v[j];
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = (uint32_t)j < mine ? (float)row[j] : -INFINITY;
        }
    }
    // The softmax's shift and sum, over all experts.
    float top = 0.0f;
    double total = 0.0;
    if (!a.sigmoid && (kWide || !a.renormalize)) {
        float m = x[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = larger(m, x[j]);
        m = join<L>(m, [](float p, float q) { return larger(p, q); });
        top = m == -INFINITY || m != m ? 0.0f : m;
    }
    // A NaN or +inf leaves the softmax no distribution.
    bool odd = false;
    if (!a.sigmoid) {
#pragma unroll
        for (int j = 0; j < V; ++j) odd = odd || !(x[j] < INFINITY);
        odd = join<L>((uint32_t)odd, [](uint32_t p, uint32_t q) { return p | q; });
    }
    S s[V];
    if constexpr (kWide) {
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = 1.0 / (1.0 + exp(-(double)x[j]));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) total += s[j] = exp((double)x[j] - (double)top);
            total = join<L>(total, [](double p, double q) { return p + q; });
            const double one = 1.0 / total;
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] *= one;
        }
        if (a.bias)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if ((uint32_t)j < mine) s[j] += (double)a.bias[first + j];
    } else {
        if (!a.sigmoid && !a.renormalize) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) sum += expf(x[j] - top);
            total = join<L>((double)sum, [](double p, double q) { return p + q; });
        }
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = x[j];
    }
    constexpr S kLowest = kWide ? (S)-1.7976931348623157e308 : (S)-3.4028234663852886e38f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (s[j] != s[j]) s[j] = kLowest;
        if (x[j] == -INFINITY) s[j] = kNone;
    }
    if (a.kept < a.groups) {
        Best<S> b{kNone, kNone};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            b.second = larger(b.second, b.first < s[j] ? b.first : s[j]);
            b.first = larger(b.first, s[j]);
        }
        if (a.group_lanes > 1) join_best<1>(b);
        if (a.group_lanes > 2) join_best<2>(b);
        if (a.group_lanes > 4) join_best<4>(b);
        if (a.group_lanes > 8) join_best<8>(b);
        if constexpr (L > 16) {
            if (a.group_lanes > 16) join_best<16>(b);
            if (a.group_lanes > 32) join_best<32>(b);
        }
        S score = b.first;
        if (a.best > 1 && b.second != kNone) score += b.second;
        uint32_t before = 0;
        for (uint32_t g = 0; g < a.groups; ++g) {
            const S other = __shfl(score, (int)(g * a.group_lanes), L);
            before += other > score || (other == score && g < group);
        }
        if (before >= a.kept)
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = kNone;
    }
    for (uint32_t i = 0; i < a.k; ++i) {
        S m = s[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = larger(m, s[j]);
        m = join<L>(m, [](S p, S q) { return larger(p, q); });
        uint32_t e = UINT32_MAX;
#pragma unroll
        for (int j = V - 1; j >= 0; --j)
            if (s[j] == m) e = first + j;
        if (m == kNone) e = UINT32_MAX;
        const uint32_t won = join<L>(e, [](uint32_t p, uint32_t q) { return lower(p, q); });
        if (won == UINT32_MAX) {
            if (lane == 0) chosen[local][i] = -1;
        } else if (won == e) {
            float at = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (won == first + j) {
                    at = x[j];
                    s[j] = kNone;
                }
            chosen[local][i] = (int32_t)won;
            chosen_x[local][i] = at;
        }
    }
    __syncthreads();
    // Lane j has the slots j, j + L, ...
    double shift = -INFINITY;
    if (a.renormalize) {
        for (uint32_t i = lane; i < a.k; i += L)
            if (chosen[local][i] >= 0) {
                const double v = a.sigmoid ? log_sigmoid(chosen_x[local][i]) : (double)chosen_x[local][i];
                if (!(v <= shift)) shift = v;  // NaN too
            }
        shift = join<L>(shift, [](double p, double q) { return q != q || q > p ? q : p; });
    }
    double weight[(kMaxK + L - 1) / L], sum = 0.0;
#pragma unroll
    for (int n = 0; n < (kMaxK + L - 1) / L; ++n) {
        const uint32_t i = lane + n * L;
        double w = 0.0;
        if (i < a.k && chosen[local][i] >= 0) {
            const double v = (double)chosen_x[local][i];
            if (a.renormalize) w = exp((a.sigmoid ? log_sigmoid(v) : v) - shift);
            else w = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / total;
        }
        weight[n] = w;
        sum += w;
    }
    double factor = odd ? (double)NAN : a.scale;
    if (a.renormalize) factor /= join<L>(sum, [](double p, double q) { return p + q; });
    if (!live) return;
#pragma unroll
    for (int n = 0; n < (kMaxK + L - 1) / L; ++n) {
        const uint32_t i = lane + n * L;
        if (i < a.k) {
            const int32_t e = chosen[local][i];
            a.experts[(int64_t)token * a.k + i] = e;
            a.weights[(int64_t)token * a.k + i] = e >= 0 ? (float)(weight[n] * factor) : 0.0f;
        }
    }
}

struct RouteGradArgs {
    int64_t stride, dstride;
    const int32_t *experts;
    const float *dweights;
    uint32_t tokens, num_experts, k;
    uint32_t sigmoid, renormalize;
    double scale;
};

// A wave a token: the chosen slots' gradients in LDS, then the row.  What the
// softmax over all experts needs is the row's maximum and sum.
template <class T>
__global__ __launch_bounds__(kOpThreads) void route_grad_kernel(const T *logits, T *dlogits,
                                                                RouteGradArgs a) {
    constexpr int kTokens = kOpThreads / 64;
    __shared__ float grad[kTokens][kMaxK];
    __shared__ int32_t expert[kTokens][kMaxK];
    const uint32_t lane = threadIdx.x % 64, local = threadIdx.x / 64;
    const uint32_t token = blockIdx.x * kTokens + local;
    const bool live = token < a.tokens;
    const T *row = logits + (int64_t)(live ? token : 0) * a.stride;
    const bool whole = !a.sigmoid && !a.renormalize;
    double m = 0.0, total = 1.0;
    if (whole) {
        float top = -INFINITY;
        for (uint32_t e = lane; e < a.num_experts; e += 64) top = larger(top, (float)row[e]);
        top = join<64>(top, [](float p, float q) { return larger(p, q); });
        m = top == -INFINITY ? 0.0 : (double)top;
        float sum = 0.0f;
        for (uint32_t e = lane; e < a.num_experts; e += 64) sum += expf((float)row[e] - (float)m);
        total = join<64>((double)sum, [](double p, double q) { return p + q; });
        if (total == 0.0) total = 1.0;  // nothing but -inf
    }
    int32_t e = live && lane < a.k ? a.experts[(int64_t)token * a.k + lane] : -1;
    if ((uint32_t)e >= a.num_experts) e = -1;
    const double x = e >= 0 ? (double)(float)row[e] : 0.0;
    const double g = e >= 0 ? a.scale * (double)a.dweights[(int64_t)token * a.k + lane] : 0.0;
    double d = 0.0;  // dlogits of the slot's expert, but for the softmax's common term
    double common = 0.0;
    if (a.renormalize) {
        // u = p / sum p, and both scorings' dx follow from log p's slope.
        double v = e < 0 ? -INFINITY : a.sigmoid ? log_sigmoid(x) : x;
        const double shift = join<64>(v, [](double p, double q) { return q != q || q > p ? q : p; });
        double u = e < 0 ? 0.0 : exp(v - shift);
        const double sum = join<64>(u, [](double p, double q) { return p + q; });
        u = e < 0 ? 0.0 : u / sum;
        const double mean = join<64>(u * g, [](double p, double q) { return p + q; });
        d = e < 0 ? 0.0 : u * (g - mean);
        if (a.sigmoid && e >= 0) d *= 1.0 / (1.0 + exp(x));  // 1 - sigmoid(x)
    } else if (a.sigmoid) {
        const double p = 1.0 / (1.0 + exp(-x));
        d = e < 0 ? 0.0 : g * p / (1.0 + exp(x));
    } else {
        const double p = e < 0 ? 0.0 : exp(x - m) / total;
        common = join<64>(p * g, [](double q, double r) { return q + r; });
        d = g * p;
    }
    grad[local][lane] = (float)d;
    expert[local][lane] = e;
    __syncthreads();
    if (!live) return;
    T *out = dlogits + (int64_t)token * a.dstride;
    for (uint32_t c = lane; c < a.num_experts; c += 64) {
        float v = 0.0f;
        if (whole) v = -(float)(exp((double)(float)row[c] - m) / total * common);
        for (uint32_t i = 0; i < a.k; ++i)
            if (expert[local][i] == (int32_t)c) v += grad[local][i];
        out[c] = (T)v;
    }
}

bool good_route(const segtopk_rows *logits, int64_t tokens, int64_t experts, int64_t k,
                int32_t scoring, double scale) {
    return tokens >= 0 && tokens < INT32_MAX && experts >= 1 && experts <= kMaxExperts && k >= 1 &&
           k <= kMaxK && k <= experts && (scoring == SEGTOPK_SOFTMAX || scoring == SEGTOPK_SIGMOID) &&
           std::isfinite(scale) && (!tokens || good_rows(logits, experts));
}

}  // namespace
}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int segtopk_route(const segtopk_route_args *args, hipStream_t stream) {
    if (!args) return SEGTOPK_INVALID_ARGUMENT;
    const segtopk_route_args &q = *args;
    if (!good_route(&q.logits, q.tokens, q.num_experts, q.k, q.scoring, q.scale) || q.groups < 1 ||
        q.groups > kMaxGroups || q.num_experts % q.groups || q.kept_groups < 1 ||
        q.kept_groups > q.groups || (q.group_best != 1 && q.group_best != 2) ||
        q.k > q.kept_groups * (q.num_experts / q.groups))
        return SEGTOPK_INVALID_ARGUMENT;
    if (q.bias && !aligned(q.bias, 4)) return SEGTOPK_INVALID_ARGUMENT;
    if (!q.tokens) return SEGTOPK_OK;
    if (!q.weights || !aligned(q.weights, 4) || !q.experts || !aligned(q.experts, 4))
        return SEGTOPK_INVALID_ARGUMENT;
    RouteArgs a{};
    a.stride = q.logits.stride;
    a.bias = q.bias;
    a.weights = q.weights;
    a.experts = q.experts;
    a.tokens = (uint32_t)q.tokens;
    a.num_experts = (uint32_t)q.num_experts;
    a.k = (uint32_t)q.k;
    // Groups that are all kept make no difference.
    a.groups = q.kept_groups == q.groups ? 1u : (uint32_t)q.groups;
    a.kept = q.kept_groups == q.groups ? 1u : (uint32_t)q.kept_groups;
    a.per_group = a.num_experts / a.groups;
    a.best = (uint32_t)q.group_best;
    a.sigmoid = q.scoring == SEGTOPK_SIGMOID;
    a.renormalize = q.renormalize != 0;
    a.scale = q.scale;
    uint32_t groups = 1;
    while (groups < a.groups) groups *= 2;
    const bool wide = a.bias || (a.groups > 1 && a.best == 2 && a.per_group > 1);
    const auto per_lane = [&](uint32_t lanes) {
        return groups > lanes ? UINT32_MAX : (a.per_group * groups + lanes - 1) / lanes;
    };
    return with_type(q.logits.type, [&](auto v) {
        using T = decltype(v);
        const T *in = static_cast<const T *>(q.logits.data);
        const auto go = [&](auto score, auto lanes, auto each) {
            constexpr int L = decltype(lanes)::value, V = decltype(each)::value;
            a.group_lanes = (uint32_t)L / groups;
            const unsigned per = kOpThreads / L;
            return status(launch(route_kernel<T, decltype(score), L, V>,
                                 dim3((a.tokens + per - 1) / per), kOpThreads, stream, 0, in, a));
        };
        const auto by_score = [&](auto lanes, auto each) {
            return wide ? go(double{}, lanes, each) : go(float{}, lanes, each);
        };
        using std::integral_constant;
        if (per_lane(16) <= 16) {
            const integral_constant<int, 16> lanes;
            const uint32_t n = per_lane(16);
            return n <= 4   ? by_score(lanes, integral_constant<int, 4>{})
                   : n <= 8 ? by_score(lanes, integral_constant<int, 8>{})
                            : by_score(lanes, integral_constant<int, 16>{});
        }
        const integral_constant<int, 64> lanes;
        const uint32_t n = per_lane(64);
        return n <= 8    ? by_score(lanes, integral_constant<int, 8>{})
               : n <= 16 ? by_score(lanes, integral_constant<int, 16>{})
                         : by_score(lanes, integral_constant<int, 32>{});
    });
}

extern "C" int segtopk_route_backward(const segtopk_rows *logits, const segtopk_rows *dlogits,
                                      const int32_t *experts, const float *dweights,
                                      int64_t tokens, int64_t num_experts, int64_t k,
                                      int32_t scoring, int32_t renormalize, double scale,
                                      hipStream_t stream) {
    if (!good_route(logits, tokens, num_experts, k, scoring, scale)) return SEGTOPK_INVALID_ARGUMENT;
    if (!tokens) return SEGTOPK_OK;
    if (!good_rows(dlogits, num_experts) || dlogits->type != logits->type || !experts ||
        !aligned(experts, 4) || !dweights || !aligned(dweights, 4))
        return SEGTOPK_INVALID_ARGUMENT;
    RouteGradArgs a{logits->stride, dlogits->stride, experts, dweights, (uint32_t)tokens,
                    (uint32_t)num_experts, (uint32_t)k, scoring == SEGTOPK_SIGMOID,
                    renormalize != 0, scale};
    return with_type(logits->type, [&](auto v) {
        using T = decltype(v);
        const unsigned per = kOpThreads / 64;
        return status(launch(route_grad_kernel<T>, dim3((a.tokens + per - 1) / per), kOpThreads,
                             stream, 0, static_cast<const T *>(logits->data),
                             static_cast<T *>(dlogits->data), a));
    });
}
