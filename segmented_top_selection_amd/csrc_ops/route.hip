// route.hip -- a router's selection from logits to gate weights, and the gradient
// of its logits.
//
//   p = softmax(x) | sigmoid(x);  s = p + bias;  the best groups by the sum of
//   their one or two best s;  the k best s of those;  w = scale p / (sum p | 1)
//
// Which experts are chosen has to be right to the last: s of two experts may be as
// near as the inputs make them.  Scores of 32 bits, as whole numbers with the expert's
// place behind them, are compared first, and settle it where all that the choice hangs
// on is further apart than they are off; else a wave compares them in 64 bits (2^-52).
// Where no bias and no sum of two scores is asked for, s orders the experts as x does,
// and x itself is compared.
//
// A token belongs to L lanes (16, so that four tokens share a wave's instructions,
// or 64), and each group of experts to a power of two of them, V neighbouring
// experts to a lane: the group's best are then found by a butterfly of a few lanes,
// and the lower index is the lower lane and the lower place in it.  The k best are
// taken one after the other, each by the largest of a lane's V and a butterfly.
//
// Bound by the vector units, 90% busy: a wave's four tokens take some 1100 instructions,
// 400 of them for eight picks and 200 for the gates in 64 bits.  32768 tokens, 8 of 256
// experts in 4 of 8 groups, f32 by the sigmoid with a bias: 21.9 us, 1.6 TB/s, against 45.5
// with all scores in 64 bits; 18.4 if no token were left for them, since all waves run at once
// and wait for the one that has such a token.  One token of 64 experts: 5.5 us a call, 4.0 of it the kernel.
#include <cmath>
#include <type_traits>

#include "ops_common.h"

namespace segtopk_ops {
namespace {

constexpr uint32_t kExpert = 1u << 31;  // marks an expert's number among keys
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

// Of numbers without NaN.
__device__ inline float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ inline double larger(double a, double b) { return a > b ? a : b; }
__device__ inline uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
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

// What a lane has of its token: its experts' logits, and where they are.
template <int V> struct Mine {
    float x[V];
    uint32_t first, count, group;
    float top;  // the softmax's shift
};

// V neighbouring numbers, of which there are `count`.
template <int V, class T>
__device__ inline void load_some(const T *from, uint32_t count, float otherwise, float *to) {
    typedef T mem __attribute__((ext_vector_type(V), aligned(sizeof(T))));
    if (count == (uint32_t)V) {
        const mem v = *reinterpret_cast<const mem *>(from);
#pragma unroll
        for (int j = 0; j < V; ++j) to[j] = (float)v[j];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) to[j] = (uint32_t)j < count ? (float)from[j] : otherwise;
    }
}
// What lane `lane` of a token's has.
template <int V, class T>
__device__ inline Mine<V> mine_of(const T *row, const RouteArgs &a, uint32_t group_lanes,
                                  uint32_t lane, bool live) {
    Mine<V> m;
    m.group = lane / group_lanes;
    const uint32_t in_group = (lane % group_lanes) * V;
    m.first = m.group * a.per_group + in_group;
    m.count = !live || m.group >= a.groups || in_group >= a.per_group ? 0u
              : a.per_group - in_group < (uint32_t)V               ? a.per_group - in_group
                                                                   : (uint32_t)V;
    load_some<V>(row + m.first, m.count, -INFINITY, m.x);
    m.top = 0.0f;
    return m;
}

// How scores are made: as the logits, or as p + bias in 32 or 64 bits.
enum { kByLogits, kBy32, kBy64 };
template <int HOW> struct ScoreType { using type = float; };
template <> struct ScoreType<kBy64> { using type = double; };

__device__ inline float exponential(float v) { return __expf(v); }
__device__ inline double exponential(double v) { return exp(v); }

// The scores of a lane's experts, whatever they are where x is -inf or NaN.
// Returns how far a score p of 32 bits is off at most: 4e-7 for the sigmoid, by its slope
// times the exponential's error, |x| 2^-24 p (1 - p) and 2^-22 p (1 - p), and its own
// roundings; 1.5e-6 of the largest p for the softmax, by the exponent's, (x - top) 2^-23 p, at
// most 0.37 of it, the exponential's, and those of a sum of up to 32 + 6 terms and a quotient.
template <int HOW, int L, int V, class S>
__device__ inline float make_scores(const Mine<V> &a, const RouteArgs &q, S *s) {
    float off = 0.0f;
    if constexpr (HOW == kByLogits) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = a.x[j];
    } else {
        if (q.sigmoid) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const S d = (S)1 + exponential(-(S)a.x[j]);
                if constexpr (HOW == kBy64) s[j] = 1.0 / d;
                else s[j] = __builtin_amdgcn_rcpf(d);
            }
            off = 4e-7f;
        } else {
            S total = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) total += s[j] = exponential((S)a.x[j] - (S)a.top);
            total = join<L>(total, [](S p, S r) { return p + r; });
            const S one = (S)1 / total;
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] *= one;
            off = 1.5e-6f * (float)one;
        }
        if (q.bias) {
            float b[V];
            load_some<V>(q.bias + a.first, a.count, 0.0f, b);
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += (S)b[j];
        }
    }
    return off;
}

// A lane's scores with what is ruled out at -inf, and a NaN at the lowest number; in 64 bits at
// -2^1022, which no score with a bias of 32 bits reaches, so that a group's two are a number
// still and not what marks a group without experts.
template <int V, class S> __device__ inline void rule_out(const Mine<V> &a, S *s) {
    constexpr S kLowest = sizeof(S) == 8 ? (S)-0x1p1022 : (S)-3.4028234663852886e38f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (s[j] != s[j]) s[j] = kLowest;
        if (a.x[j] == -INFINITY) s[j] = (S)-INFINITY;
    }
}

// What lane `lane` of the token's has; the wave's own is a scalar.
template <int L> __device__ inline float score_of(float score, uint32_t lane) {
    if constexpr (L < 64) return __shfl(score, (int)lane, L);
    else return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(score), (int)lane));
}
template <int L> __device__ inline double score_of(double score, uint32_t lane) {
    if constexpr (L < 64) return __shfl(score, (int)lane, L);
    else return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(score), (int)lane),
                                 __builtin_amdgcn_readlane(__double2loint(score), (int)lane));
}
// Rules out the experts of groups that are not kept.  With `off` (scores of 32 bits): whether
// scores so far off, and by their sum's rounding, could make another choice.
template <int L, int V, class S>
__device__ inline bool keep_groups(const Mine<V> &a, const RouteArgs &q, S *s, float off) {
    constexpr S kNone = (S)-INFINITY;
    constexpr float kMost = 3.4028234663852886e38f;
    if (q.kept >= q.groups) return false;
    Best<S> b{kNone, kNone};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        b.second = larger(b.second, b.first < s[j] ? b.first : s[j]);
        b.first = larger(b.first, s[j]);
    }
    if (q.group_lanes > 1) join_best<1>(b);
    if (q.group_lanes > 2) join_best<2>(b);
    if (q.group_lanes > 4) join_best<4>(b);
    if (q.group_lanes > 8) join_best<8>(b);
    if constexpr (L > 16) {
        if (q.group_lanes > 16) join_best<16>(b);
        if (q.group_lanes > 32) join_best<32>(b);
    }
    S score = b.first;
    if (q.best > 1 && b.second != kNone) score += b.second;
    // Scores of 32 bits whose sum leaves them stay at their end, where they are near each other:
    // -inf marks a group without experts, and nothing is near an infinity.
    if (off > 0.0f && b.first != kNone) score = larger((S)-kMost, score < (S)kMost ? score : (S)kMost);
    uint32_t before = 0;
    bool unsure = false;
    if (off > 0.0f) {
        // Two sums of two scores, each off by that, by a bias's rounding and its own.
        const S most = join<L>(score == kNone ? (S)0 : (S)fabsf((float)score),
                               [](S p, S r) { return larger(p, r); });
        const S by = (S)4 * (S)off + (S)0x1p-20 * most;
        const S over = score + by, under = score - by;
        uint32_t perhaps = 0;  // its own too
        for (uint32_t g = 0; g < q.groups; ++g) {
            const S other = score_of<L>(score, g * q.group_lanes);
            before += other > over;
            perhaps += other >= under;
        }
        unsure = a.group < q.groups && score != kNone && before < q.kept && perhaps > q.kept;
    } else {
        for (uint32_t g = 0; g < q.groups; ++g) {
            const S other = score_of<L>(score, g * q.group_lanes);
            before += other > score || (other == score && g < a.group);
        }
    }
    if (before >= q.kept)
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = kNone;
    return unsure;
}

// The k best by comparing scores, equal ones by their index, by a whole wave.  A batch's waves
// may all run at once, and one such token is then the last to be done.
template <int HOW, int V>
__device__ inline void choose_exactly(const Mine<V> &a, const RouteArgs &q, uint32_t *chosen) {
    using S = typename ScoreType<HOW>::type;
    constexpr S kNone = (S)-INFINITY;
    S s[V];
    make_scores<HOW, 64>(a, q, s);
    rule_out<V>(a, s);
    keep_groups<64>(a, q, s, 0.0f);
#pragma unroll 1
    for (uint32_t i = 0; i < q.k; ++i) {
        S m = s[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = larger(m, s[j]);
        const S own = m;
        m = join<64>(m, [](S p, S r) { return larger(p, r); });
        // The lowest lane's lowest place.
        const int first = __builtin_ctzll(__ballot(own == m));
        uint32_t e = 0;
#pragma unroll
        for (int j = V - 1; j >= 0; --j)
            if (s[j] == m) e = a.first + j;
        const uint32_t won = m == kNone ? UINT32_MAX : (uint32_t)__builtin_amdgcn_readlane((int)e, first);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (won == a.first + j) s[j] = kNone;
        if (threadIdx.x % 64 == 0) chosen[i] = kExpert | won;
    }
}

// The k best by keys that no two experts share: the score in the high bits, 0 for what is
// ruled out, and the place among the token's lanes in the low ones, the first place highest.
// The next best is the largest key below the last: key - last, as an unsigned number, is the
// larger the nearer the key is below, and under 2^31 where it is not below.  A step is a
// subtraction and half a maximum of three for each expert.
// Returns whether two scores that the choice hangs on are within `near` of each other.
template <int L, int V>
__device__ inline bool choose_by_keys(const uint32_t *key, const RouteArgs &q, uint32_t near,
                                      bool inexact, uint32_t *chosen) {
    constexpr int kBits = __builtin_ctz(L * V);
    bool unsure = false;
    uint32_t last = 1u << 31;
#pragma unroll 1
    for (uint32_t i = 0; i < q.k + (inexact ? 1u : 0u); ++i) {
        uint32_t below = key[0] - last;
#pragma unroll
        for (int j = 1; j < V; ++j) below = larger(below, key[j] - last);
        below = join<L>(below, [](uint32_t p, uint32_t r) { return larger(p, r); });
        const uint32_t next = last ? last + below : 0u;
        unsure = unsure || (i && next >> kBits && (last >> kBits) - (next >> kBits) <= near);
        last = next;
        if (i < q.k && threadIdx.x % L == 0) chosen[i] = next;
    }
    return inexact && unsure;
}
// The expert of what has been chosen, -1: none.
template <int L, int V> __device__ inline int32_t expert_of(uint32_t chosen, const RouteArgs &q) {
    constexpr uint32_t kPlaces = L * V;
    if (chosen & kExpert) return chosen == UINT32_MAX ? -1 : (int32_t)(chosen & ~kExpert);
    if (chosen < kPlaces) return -1;
    const uint32_t place = kPlaces - 1 - chosen % kPlaces, lane = place / V;
    const uint32_t group = lane >> __builtin_ctz(q.group_lanes);  // a power of two
    const uint32_t expert = group * q.per_group + (lane & (q.group_lanes - 1)) * V + place % V;
    // Its logit is loaded: no key may lead out of the row.
    return expert < q.num_experts ? (int32_t)expert : -1;
}

// The k best by scores of 32 bits, as whole numbers over the range of the token's scores.
template <int HOW, int L, int V>
__device__ inline bool choose_nearly(const Mine<V> &a, const RouteArgs &q, uint32_t *chosen) {
    constexpr int kPlaces = L * V, kBits = __builtin_ctz(kPlaces);
    constexpr float kSteps = (float)((1u << (31 - kBits)) - 8u);
    float s[V];
    const float off = make_scores<HOW, L>(a, q, s);
    // These keep NaN.
    float high = s[0], low = s[0], least = a.x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) {
        high = larger(high, s[j]);
        low = __builtin_elementwise_minimum(low, s[j]);
        if constexpr (HOW != kByLogits) least = __builtin_elementwise_minimum(least, a.x[j]);
    }
    // Where none of a wave's scores is ruled out or NaN, nobody looks at each for that.
    const bool clean = !__any(!(high < INFINITY) || !(low > -INFINITY) || !(least > -INFINITY));
    if (!clean) {
        rule_out<V>(a, s);
        high = low = -INFINITY;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            high = larger(high, s[j]);
            const float v = s[j] == -INFINITY ? INFINITY : s[j];
            low = j ? fminf(low, v) : v;
        }
    }
    high = join<L>(high, [](float p, float r) { return larger(p, r); });
    low = join<L>(low, [](float p, float r) { return fminf(p, r); });
    const bool unsure = keep_groups<L>(a, q, s, HOW == kBy32 ? off : 0.0f);
    // Nothing but one number, or numbers too near each other or too far apart to be told by
    // finite steps: all of them count as near each other.  kSteps is below 2^25, so that steps
    // are below 2^125 and no number comes to more than kSteps and 2, or bit 31 of a key.
    const float range = high - low;
    const float steps = range >= 0x1p-100f ? kSteps / range : 0.0f;
    uint32_t key[V];
    const uint32_t place = threadIdx.x % L * V;
    if (clean && !__any(steps == 0.0f)) {
#pragma unroll
        for (int j = 0; j < V; ++j)  // groups that are not kept become 0
            key[j] = (uint32_t)fmaxf(fmaf(s[j] - low, steps, 1.0f), 0.0f) << kBits | (kPlaces - 1 - place - j);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t n = 1u + (uint32_t)((s[j] == -INFINITY ? 0.0f : s[j] - low) * steps);
            key[j] = s[j] == -INFINITY ? 0u : n << kBits | (kPlaces - 1 - place - j);
        }
    }
    // Each is off by `off` and by the bias's rounding, and by less than 2 steps in the product.
    const float by = 2.0f * off + 0x1p-22f * (fabsf(high) + fabsf(low));
    const uint32_t near = HOW == kBy32 ? (uint32_t)fminf(by * steps, 1e9f) + 4u : 4u;
    return choose_by_keys<L, V>(key, q, near, true, chosen) || unsure;
}

// The k best by logits of 16 bits, whose order is that of whole numbers.
template <class T, int L, int V>
__device__ inline void choose_by_16(const Mine<V> &a, const RouteArgs &q, uint32_t *chosen) {
    constexpr int kPlaces = L * V, kBits = __builtin_ctz(kPlaces);
    static_assert(kBits + 17 <= 31, "");
    float s[V];
    make_scores<kByLogits, L>(a, q, s);
    rule_out<V>(a, s);
    keep_groups<L>(a, q, s, 0.0f);
    uint32_t key[V];
    const uint32_t place = threadIdx.x % L * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        // The zeros are equal, and the lowest number stands for NaN.
        const float v = larger(s[j] + 0.0f, std::is_same<T, __bf16>::value ? -3.3895313892515355e38f : -65504.0f);
        const uint32_t bits = __builtin_bit_cast(uint16_t, (T)v);
        const uint32_t order = (bits & 0x8000u ? 0xFFFFu - bits : bits + 0x8000u) + 1u;
        key[j] = s[j] == -INFINITY ? 0u : order << kBits | (kPlaces - 1 - place - j);
    }
    choose_by_keys<L, V>(key, q, 0, false, chosen);
}

template <class T, bool BY_LOGITS, int L, int V>
__global__ __launch_bounds__(kOpThreads) void route_kernel(const T *logits, RouteArgs a) {
    constexpr int kTokens = kOpThreads / L;
    __shared__ uint32_t chosen[kTokens][kMaxK];
    const uint32_t lane = threadIdx.x % L, local = threadIdx.x / L;
    const uint32_t token = blockIdx.x * kTokens + local;
    // All lanes of a wave stay for the butterflies; lanes without a token have none to choose from.
    const bool live = token < a.tokens;
    const T *const row = logits + (int64_t)(live ? token : 0) * a.stride;
    Mine<V> mine = mine_of<V>(row, a, a.group_lanes, lane, live);
    // The softmax's shift and sum, over all experts; a NaN or +inf leaves it no distribution.
    double total = 0.0;
    bool odd = false;
    if (!a.sigmoid) {
        float m = mine.x[0];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            m = fmaxf(m, mine.x[j]);
            odd = odd || !(mine.x[j] < INFINITY);
        }
        odd = join<L>((uint32_t)odd, [](uint32_t p, uint32_t q) { return p | q; });
        m = join<L>(m, [](float p, float q) { return fmaxf(p, q); });
        mine.top = m == -INFINITY || odd ? 0.0f : m;
        if (!a.renormalize) {
            // A sum of 32 bits leaves a weight 3.2 half steps of 32 bits off (seen on normal
            // logits), one of 64 leaves it half a step: 32768 tokens, 8 of 256 in f32, 17.1 and
            // 20.2 us, 8192 of 1000 in bf16 16.5 and 19.4.  The choice does not hang on it.
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) sum += expf(mine.x[j] - mine.top);
            total = join<L>((double)sum, [](double p, double q) { return p + q; });
        }
    }
    // In 32 bits first, which nearly always settles it.
    if constexpr (BY_LOGITS && sizeof(T) == 2) {
        choose_by_16<T, L, V>(mine, a, chosen[local]);
    } else {
        constexpr int kNearly = BY_LOGITS ? kByLogits : kBy32, kExactly = BY_LOGITS ? kByLogits : kBy64;
        const bool unsure = choose_nearly<kNearly, L, V>(mine, a, chosen[local]);
        // The whole wave for each token that is not settled.
        for (uint64_t left = __ballot(unsure && live); left;) {
            const uint32_t which = (uint32_t)__builtin_ctzll(left) / L;  // of the wave's tokens
            left &= ~((L == 64 ? ~0ull : (1ull << (L % 64)) - 1) << which * L % 64);
            const uint32_t there = threadIdx.x / 64 * (64 / L) + which;
            constexpr int kFew = V * L / 64;
            RouteArgs wave = a;
            wave.group_lanes = a.group_lanes * (64 / L);
            Mine<kFew> m = mine_of<kFew>(logits + (int64_t)(blockIdx.x * kTokens + there) * a.stride, a,
                                         wave.group_lanes, threadIdx.x % 64, true);
            m.top = __shfl(mine.top, (int)(which * L));
            choose_exactly<kExactly, kFew>(m, wave, chosen[there]);
        }
    }
    __syncthreads();
    // Lane j has the slots j, j + L, ...
    constexpr int kSlots = (kMaxK + L - 1) / L;
    double x[kSlots], shift = -INFINITY, sum = 0.0;
    int32_t expert[kSlots];
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
        const uint32_t i = lane + n * L;
        expert[n] = i < a.k ? expert_of<L, V>(chosen[local][i], a) : -1;
        x[n] = expert[n] >= 0 ? (double)(float)row[expert[n]] : 0.0;
    }
    if (a.renormalize) {
        // Sigmoids that underflow are compared by their logarithms.
        bool far = false;
        if (a.sigmoid) {
#pragma unroll
            for (int n = 0; n < kSlots; ++n) far = far || (expert[n] >= 0 && x[n] < -300.0);
            far = __ballot(far);
        }
        if (!a.sigmoid || far) {
#pragma unroll
            for (int n = 0; n < kSlots; ++n) {
                if (n * L >= a.k) continue;
                if (far) x[n] = log_sigmoid(x[n]);
                if (expert[n] >= 0 && !(x[n] <= shift)) shift = x[n];  // NaN too
            }
            shift = join<L>(shift, [](double p, double q) { return q != q || q > p ? q : p; });
#pragma unroll
            for (int n = 0; n < kSlots; ++n)
                if (n * L < a.k) x[n] = exp(x[n] - shift);
        } else {
#pragma unroll
            for (int n = 0; n < kSlots; ++n)
                if (n * L < a.k) x[n] = 1.0 / (1.0 + exp(-x[n]));
        }
    } else {
#pragma unroll
        for (int n = 0; n < kSlots; ++n)
            if (n * L < a.k)
                x[n] = a.sigmoid ? 1.0 / (1.0 + exp(-x[n])) : exp(x[n] - (double)mine.top) / total;
    }
#pragma unroll
    for (int n = 0; n < kSlots; ++n)
        if (expert[n] >= 0) sum += x[n];
    double factor = odd ? (double)NAN : a.scale;
    if (a.renormalize) factor /= join<L>(sum, [](double p, double q) { return p + q; });
    if (!live) return;
#pragma unroll
    for (int n = 0; n < kSlots; ++n) {
        const uint32_t i = lane + n * L;
        if (i < a.k) {
            a.experts[(int64_t)token * a.k + i] = expert[n];
            a.weights[(int64_t)token * a.k + i] = expert[n] >= 0 ? (float)(x[n] * factor) : 0.0f;
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

// A wave a token: the chosen slots' gradients in LDS, then the row.  The softmax over all experts
// needs the row's maximum, sum and mean of g first, and is in 64 bits up to one rounding: of a
// router that is sure, p (g - mean) of the chosen expert is what little p leaves to the others,
// and 32 bits would have nothing of it left from 1 - p = 2^-24 on (8192 tokens, 8 of 128 in
// bf16, 8.2 -> 8.7 us a call).  Elsewhere nothing cancels behind the slots' own 64 bits.
template <class T>
__global__ __launch_bounds__(kOpThreads) void route_grad_kernel(const T *logits, T *dlogits,
                                                                RouteGradArgs a) {
    constexpr int kTokens = kOpThreads / 64;
    __shared__ float grad[kTokens][kMaxK];
    __shared__ double given[kTokens][kMaxK];  // g, for the softmax over all
    __shared__ int32_t expert[kTokens][kMaxK];
    const uint32_t lane = threadIdx.x % 64, local = threadIdx.x / 64;
    const uint32_t token = blockIdx.x * kTokens + local;
    const bool live = token < a.tokens;
    const T *row = logits + (int64_t)(live ? token : 0) * a.stride;
    const bool whole = !a.sigmoid && !a.renormalize;
    double m = 0.0, total = 1.0;
    if (whole) {
        float top = -INFINITY;
        for (uint32_t e = lane; e < a.num_experts; e += 64) top = fmaxf(top, (float)row[e]);
        top = join<64>(top, [](float p, float q) { return fmaxf(p, q); });
        m = top == -INFINITY ? 0.0 : (double)top;
        double sum = 0.0;
        for (uint32_t e = lane; e < a.num_experts; e += 64) sum += exp((double)(float)row[e] - m);
        total = join<64>(sum, [](double p, double q) { return p + q; });
        if (total == 0.0) total = 1.0;  // nothing but -inf
    }
    int32_t e = live && lane < a.k ? a.experts[(int64_t)token * a.k + lane] : -1;
    if ((uint32_t)e >= a.num_experts) e = -1;
    const double x = e >= 0 ? (double)(float)row[e] : 0.0;
    const double g = e >= 0 ? a.scale * (double)a.dweights[(int64_t)token * a.k + lane] : 0.0;
    double d = 0.0;     // dlogits of the slot's expert
    double mean = 0.0;  // of g, by p
    if (a.renormalize) {
        // u = p / sum p, and both scorings' dx follow from log p's slope.
        double v = e < 0 ? -INFINITY : a.sigmoid ? log_sigmoid(x) : x;
        const double shift = join<64>(v, [](double p, double q) { return q != q || q > p ? q : p; });
        double u = e < 0 ? 0.0 : exp(v - shift);
        const double sum = join<64>(u, [](double p, double q) { return p + q; });
        u = e < 0 ? 0.0 : u / sum;
        mean = join<64>(u * g, [](double p, double q) { return p + q; });
        d = e < 0 ? 0.0 : u * (g - mean);
        if (a.sigmoid && e >= 0) d *= 1.0 / (1.0 + exp(x));  // 1 - sigmoid(x)
    } else if (a.sigmoid) {
        const double p = 1.0 / (1.0 + exp(-x));
        d = e < 0 ? 0.0 : g * p / (1.0 + exp(x));
    } else {
        const double p = e < 0 ? 0.0 : exp(x - m) / total;
        mean = join<64>(p * g, [](double q, double r) { return q + r; });
        given[local][lane] = g;
    }
    grad[local][lane] = (float)d;
    expert[local][lane] = e;
    __syncthreads();
    if (!live) return;
    T *out = dlogits + (int64_t)token * a.dstride;
    for (uint32_t c = lane; c < a.num_experts; c += 64) {
        float v = 0.0f;
        if (whole) {
            double own = 0.0;
            for (uint32_t i = 0; i < a.k; ++i)
                if (expert[local][i] == (int32_t)c) own += given[local][i];
            v = (float)(exp((double)(float)row[c] - m) / total * (own - mean));
        } else {
            for (uint32_t i = 0; i < a.k; ++i)
                if (expert[local][i] == (int32_t)c) v += grad[local][i];
        }
        out[c] = (T)v;
    }
}

bool good_route(const segtopk_rows *logits, int64_t tokens, int64_t experts, int64_t k,
                int32_t scoring, double scale) {
    return tokens >= 0 && tokens < INT32_MAX && experts >= 1 && experts <= kMaxExperts && k >= 1 &&
           k <= kMaxK && k <= experts && (scoring == SEGTOPK_SOFTMAX || scoring == SEGTOPK_SIGMOID) &&
           std::isfinite(scale) && (!tokens || good_rows(logits, experts));
}
constexpr int64_t kMostTokens = kMostBlocks * (kOpThreads / 64);  // a wave each

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
    if (q.tokens > kMostTokens) return SEGTOPK_NOT_SUPPORTED;
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
            return status(launch(route_kernel<T, decltype(score)::value, L, V>,
                                 dim3((a.tokens + per - 1) / per), kOpThreads, stream, 0, in, a));
        };
        const auto by_score = [&](auto lanes, auto each) {
            return wide ? go(std::false_type{}, lanes, each) : go(std::true_type{}, lanes, each);
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
    if (tokens > kMostTokens) return SEGTOPK_NOT_SUPPORTED;
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
