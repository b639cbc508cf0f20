// policy_loss.hip -- the clipped policy loss with a KL term, over the logits of
// sampled tokens, and its gradient.
//
// For a row t with sampled token y, z = logits / temperature:
//   lp   = z[y] - m - log sum exp(z - m),   m = max z
//   r    = exp(lp - old),  A the advantage
//   term = -min(r A, clamp(r, 1 - low, 1 + high) A)
//          + kl (exp(ref - lp) - (ref - lp) - 1)
//   loss = sum_t weight_t term_t,  weight_t = 1 / (answers * live rows of its answer)
//   d term / d lp = -(r A where the unclipped side is the minimum, else 0)
//                   + kl (1 - exp(ref - lp))
//   dlogits[c] = weight_t (d term / d lp) (1[c = y] - exp(z[c] - lse)) / temperature
// A row without a token in [0, vocab), or in no answer, counts for nothing: its
// gradient is zero.  NaN in what any other row is made of, and a logit of +inf,
// give a loss and a gradient of that row that are NaN.
//
//   count_kernel  one workgroup an answer: the number of its live rows
//   row_kernel    one workgroup a row: maximum and sum in one pass, then, where
//                 asked for, the gradient in a second that walks the row back
//                 from its end, the last pieces of it still in registers.  The
//                 last row to arrive adds up the terms, in one fixed order.
//
// The terms of a loss cancel, so each has to be better than the plain 32 bits
// that its size suggests: exponents are taken from the row's maximum, with the
// factor log2(e) / temperature in two parts, and everything after the sum, once a
// row, is in 64 bits (relative error of the loss on random cases 2e-9 to 1e-7;
// wholly in 32 bits up to 1e-5).
//
// Bound by memory where rows are many: 4096 x 131072 bf16 with its gradient, a
// quarter of the rows left out, take 366 us, 5.1 TB/s of what has to be read and
// written; by latency where they are few, a workgroup to a row: 96 x 32003 f16
// 10 us, of which the arrival takes 1 and the 64 bits 0.4.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "ops_common.h"

namespace segtopk_ops {
namespace {

struct LossArgs {
    int64_t stride, dstride;
    const void *token_ids;
    const float *old_logp, *ref_logp, *advantages;
    float *logp, *loss;
    const uint32_t *live;  // [tokens], 0 for a row that counts for nothing
    double *term;          // [tokens]
    uint32_t *arrived;
    uint32_t tokens, vocab, wide;
    double answers, clip_low, clip_high, kl_coef, temperature, grad_scale;
    float factor, rest;  // log2(e) / temperature
};

__device__ inline int64_t token_of(const void *ids, uint32_t wide, uint32_t t) {
    return wide ? static_cast<const int64_t *>(ids)[t]
                : (int64_t) static_cast<const int32_t *>(ids)[t];
}

constexpr uint32_t kCountThreads = 1024;
constexpr int64_t kCountBlocks = 1 << 16;  // of a launch; further answers in turn

// Rows arrive at one of 64 counters, and the last row of each at the counter
// before them: additions to one word follow each other 14 ns apart, which took
// 59 us of 4096 rows whatever their length.  Each has a cache line to itself.
constexpr uint32_t kCounters = 64, kCounterWords = 32;
__device__ inline uint32_t arrive(uint32_t *counter) {
    return __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(kCountThreads) void count_kernel(const void *ids, uint32_t wide,
                                                           uint32_t tokens, uint32_t vocab,
                                                           const int64_t *offsets,
                                                           uint32_t segments, uint32_t *live,
                                                           uint32_t *arrived) {
    __shared__ uint32_t total;
    const auto at = [&](uint32_t s) {  // offsets outside the rows are cut
        const int64_t v = offsets[s];
        return (uint32_t)(v < 0 ? 0 : v > (int64_t)tokens ? (int64_t)tokens : v);
    };
    const auto named = [&](int64_t y) { return y >= 0 && y < (int64_t)vocab; };
    if (blockIdx.x == 0) {  // the counters, and the rows outside every answer
        if (threadIdx.x <= kCounters) arrived[threadIdx.x * kCounterWords] = 0u;
        const uint32_t b = segments ? at(0) : tokens, e = segments ? at(segments) : tokens;
        for (uint32_t t = threadIdx.x; t < b; t += kCountThreads) live[t] = 0u;
        for (uint32_t t = e + threadIdx.x; t < tokens; t += kCountThreads) live[t] = 0u;
    }
    for (uint32_t s = blockIdx.x; s < segments; s += gridDim.x) {
        const uint32_t b = at(s), e = at(s + 1);
        if (threadIdx.x == 0) total = 0u;
        __syncthreads();
        uint32_t n = 0;
        for (uint32_t t0 = b + threadIdx.x; t0 < e; t0 += 4u * kCountThreads) {
            int64_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t t = t0 + j * kCountThreads;
                y[j] = t < e ? token_of(ids, wide, t) : -1;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) n += named(y[j]);
        }
        if (n) atomicAdd(&total, n);
        __syncthreads();
        n = total;
        for (uint32_t t = b + threadIdx.x; t < e; t += kCountThreads)
            live[t] = named(token_of(ids, wide, t)) ? n : 0u;
        __syncthreads();
    }
}

constexpr double kLog2e = 1.44269504088896340736;
constexpr int kAtOnce = 4;  // pieces of a thread that are in flight together

// Running maximum m and sum of 2^((x - m) factor).
struct Stat {
    float m, s;
};
__device__ inline float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }

// 2^(d log2(e) / temperature) for d <= 0.  `rest` is positive, so -inf gives 0.
// The hardware's exponential takes what is below 2^-126 to zero, next to a sum of
// at least one.
__device__ inline float power(float d, const LossArgs &a) {
    return __builtin_amdgcn_exp2f(fmaf(d, a.rest, d * a.factor));
}

// The statistics of 16 lanes or a whole wave as one.
template <int LANES> __device__ inline Stat join_lanes(Stat x, const LossArgs &a) {
    float m = x.m;
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    float s = x.s * power(x.m - shift_of(m), a);
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) s += __shfl_xor(s, d);
    return {m, s};
}

struct RowTail {
    float m, log2_sum, slope;
};

template <class T, bool GRAD, bool STREAM, int THREADS>
__global__ __launch_bounds__(THREADS) void row_kernel(const T *logits, T *dlogits, LossArgs a) {
    using P = Piece<T>;
    constexpr int kWaves = THREADS / 64;
    constexpr uint32_t kGroup = THREADS * kAtOnce;  // pieces
    __shared__ Stat part[16];
    __shared__ RowTail tail;
    __shared__ uint32_t arrival;
    __shared__ double sums[kWaves];
    const uint32_t t = blockIdx.x, i = threadIdx.x;
    const uint32_t live = a.live[t], token = (uint32_t)token_of(a.token_ids, a.wide, t);
    const float adv32 = a.advantages[t], old = a.old_logp[t];
    const float ref = a.kl_coef != 0.0 ? a.ref_logp[t] : 0.0f;
    const T *row = logits + (int64_t)t * a.stride;
    T *grad = GRAD ? dlogits + (int64_t)t * a.dstride : nullptr;
    const uint32_t pieces = a.vocab / P::N, groups = (pieces + kGroup - 1) / kGroup;
    const uint32_t single = pieces * P::N + i;  // the element past the pieces that is this thread's
    const T none = (T)-INFINITY;
    typename P::vec v[kAtOnce];
    T x1 = none;
    uint32_t mine = 0;
    double lp = 0.0, term = 0.0;  // of thread 0
    if (live) {
        const float xy = (float)row[token];  // read before the gradient may overwrite it
        if (single < a.vocab) x1 = row[single];
        Stat st{-INFINITY, 0.0f};
        for (uint32_t g = 0; g < groups; ++g) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const uint32_t u = g * kGroup + j * THREADS + i;
                v[j] = (typename P::vec)none;
                if (u < pieces) v[j] = load_piece(row + (size_t)u * P::N);
            }
            float m = st.m;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const typename P::f32 x = widen<T>(v[j]);
#pragma unroll
                for (int k = 0; k < P::N; ++k) m = fmaxf(m, x[k]);
            }
            const float o = shift_of(m);
            st.s *= power(st.m - o, a);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const typename P::f32 x = widen<T>(v[j]);
#pragma unroll
                for (int k = 0; k < P::N; ++k) st.s += power(x[k] - o, a);
            }
            st.m = m;
        }
        {
            const float x = (float)x1, m = fmaxf(st.m, x), o = shift_of(m);
            st.s = st.s * power(st.m - o, a) + power(x - o, a);
            st.m = m;
        }
        st = join_lanes<64>(st, a);
        if ((i & 63u) == 0) part[i >> 6] = st;
        __syncthreads();
        if (i < 64u) {
            st = part[i % kWaves];
            st = join_lanes<kWaves>(st, a);
            if (i == 0) {
                double d = 0.0;
                // Nothing but -inf: no distribution, and no loss.
                if (st.m != -INFINITY || st.s != 0.0f) {
                    lp = ((double)xy - (double)st.m) / a.temperature - log((double)st.s);
                    // Comparisons with NaN are false: it takes the side that is not
                    // clipped, and so reaches the term and the gradient.
                    const double adv = adv32, ratio = exp(lp - (double)old);
                    const double low = 1.0 - a.clip_low, high = 1.0 + a.clip_high;
                    const double clipped = ratio < low ? low : ratio > high ? high : ratio;
                    // No advantage is nothing, at a ratio past the range too.
                    const bool nothing = adv == 0.0 && ratio == INFINITY;
                    const double gain = nothing ? 0.0 : ratio * adv;
                    const double bound = nothing ? 0.0 : clipped * adv;
                    const bool held = gain > bound;
                    term = held ? -bound : -gain;
                    d = held ? 0.0 : -gain;
                    if (a.kl_coef != 0.0) {
                        const double apart = (double)ref - lp, e = exp(apart);
                        // Infinite where a token ruled out was sampled: apart is, too.
                        term += a.kl_coef * (e == INFINITY ? e : e - apart - 1.0);
                        d += a.kl_coef * (1.0 - e);
                    }
                    const double weight = 1.0 / (a.answers * (double)live);
                    term *= weight;
                    d *= weight / a.temperature * a.grad_scale;
                }
                tail = {shift_of(st.m), log2f(st.s), (float)d};
            }
        }
    }
    if (GRAD) __syncthreads();
    if (i == 0) {
        a.logp[t] = (float)lp;
        __hip_atomic_store(&a.term[t], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // The term is stored past this XCD's cache, and has arrived where every
        // XCD sees it before the row counts as arrived.  A release at device
        // scope would do so by writing the whole cache back, the gradient with
        // it, once a row: 638 us for 4096 x 131072 bf16 where this takes 366.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        mine = arrive(a.arrived + (1u + t % kCounters) * kCounterWords);
    }
    if (GRAD) {
        const float slope = live ? tail.slope : 0.0f, m = tail.m, l = tail.log2_sum;
        if (slope == 0.0f) {
            for (uint32_t u = i; u < pieces; u += THREADS)
                store_piece<STREAM>(grad + (size_t)u * P::N, (typename P::vec)(T)0.0f);
            if (single < a.vocab) grad[single] = (T)0.0f;
        } else if (fabsf(slope) == INFINITY) {
            // Of a token ruled out: infinite, but zero where no probability moves.
            for (uint32_t c = i; c < a.vocab; c += THREADS) {
                const float p = __builtin_amdgcn_exp2f(fmaf((float)row[c] - m, a.factor, -l));
                const float moves = (c == token ? 1.0f : 0.0f) - p;
                grad[c] = (T)(moves == 0.0f ? 0.0f : slope * moves);
            }
        } else {
            const uint32_t hot = token / P::N, place = token % P::N;
            for (uint32_t g = groups; g-- > 0;) {
                if (g + 1 < groups) {
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j) {
                        const uint32_t u = g * kGroup + j * THREADS + i;  // below pieces
                        v[j] = load_piece<STREAM>(row + (size_t)u * P::N);
                    }
                }
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const uint32_t u = g * kGroup + j * THREADS + i;
                    if (u >= pieces) continue;
                    const typename P::f32 x = widen<T>(v[j]);
                    typename P::f32 d;
#pragma unroll
                    for (int k = 0; k < P::N; ++k)
                        d[k] = -slope * __builtin_amdgcn_exp2f(fmaf(x[k] - m, a.factor, -l));
                    if (u == hot)
#pragma unroll
                        for (int k = 0; k < P::N; ++k)
                            if ((uint32_t)k == place) d[k] += slope;
                    store_piece<STREAM>(grad + (size_t)u * P::N, narrow<T>(d));
                }
            }
            if (single < a.vocab) {
                const float p = __builtin_amdgcn_exp2f(fmaf((float)x1 - m, a.factor, -l));
                grad[single] = (T)(slope * ((single == token ? 1.0f : 0.0f) - p));
            }
        }
    }
    if (i == 0) {
        const uint32_t of_its_counter = (a.tokens - 1u - t % kCounters) / kCounters + 1u;
        arrival = mine + 1u == of_its_counter ? arrive(a.arrived) : kCounters;
    }
    __syncthreads();
    if (arrival + 1u != min(a.tokens, kCounters)) return;
    // Every other row's term is there.
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    double sum = 0.0;
    for (uint32_t r = i; r < a.tokens; r += THREADS)
        sum += __hip_atomic_load(&a.term[r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if ((i & 63u) == 0) sums[i >> 6] = sum;
    __syncthreads();
    if (i == 0) {
        for (int w = 1; w < kWaves; ++w) sum += sums[w];
        *a.loss = (float)sum;
    }
}

__global__ void no_rows_kernel(float *loss) { *loss = 0.0f; }

size_t term_bytes(int64_t tokens) { return ((size_t)tokens * 8 + 255) & ~(size_t)255; }

size_t live_bytes(int64_t tokens) { return ((size_t)tokens * 4 + 255) & ~(size_t)255; }

// The terms, the live counts, and the counters of arrivals.
size_t loss_workspace(int64_t tokens) {
    return tokens ? term_bytes(tokens) + live_bytes(tokens) + (1 + kCounters) * kCounterWords * 4 : 0;
}

bool good_loss_sizes(int64_t tokens, int64_t vocab, int64_t segments) {
    // One workgroup of 1024 threads a row, fewer than 2^32 threads in all.
    return tokens >= 0 && tokens < (1 << 22) && vocab >= 1 && vocab <= INT32_MAX &&
           segments >= 0 && segments < (1 << 24);
}

}  // namespace
}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int64_t segtopk_policy_loss_workspace(int64_t tokens, int64_t vocab,
                                                 int64_t num_segments) {
    if (!good_loss_sizes(tokens, vocab, num_segments)) return 0;
    return (int64_t)loss_workspace(tokens);
}

extern "C" int segtopk_policy_loss(const segtopk_policy_loss_args *args, void *workspace,
                                   int64_t workspace_bytes, hipStream_t stream) {
    if (!args) return SEGTOPK_INVALID_ARGUMENT;
    const segtopk_policy_loss_args &q = *args;
    if (!good_loss_sizes(q.tokens, q.vocab, q.num_segments)) return SEGTOPK_INVALID_ARGUMENT;
    const bool grad = q.dlogits.data != nullptr;
    const int ib = index_bytes(q.id_type);
    // The comparisons are false for NaN, which is refused with the rest.
    if (!(q.clip_low >= 0.0 && q.clip_low <= 1.0) || !(q.clip_high >= 0.0) ||
        !(q.kl_coef >= 0.0) || !(q.temperature > 0.0) || !(q.temperature < INFINITY) ||
        !(q.grad_scale - q.grad_scale == 0.0) || !(q.kl_coef < INFINITY) || !ib)
        return SEGTOPK_INVALID_ARGUMENT;
    if (!q.loss || !aligned(q.loss, 4)) return SEGTOPK_INVALID_ARGUMENT;
    if (q.num_segments && (!q.segment_offsets || !aligned(q.segment_offsets, 8)))
        return SEGTOPK_INVALID_ARGUMENT;
    if (q.tokens) {
        if (!good_rows(&q.logits, q.vocab) || !q.token_ids || !aligned(q.token_ids, ib) ||
            !q.old_logp || !aligned(q.old_logp, 4) || !q.advantages || !aligned(q.advantages, 4) ||
            !q.logp || !aligned(q.logp, 4) || !aligned(q.ref_logp, 4) ||
            (q.kl_coef != 0.0 && !q.ref_logp))
            return SEGTOPK_INVALID_ARGUMENT;
        if (grad && (!good_rows(&q.dlogits, q.vocab) || q.dlogits.type != q.logits.type))
            return SEGTOPK_INVALID_ARGUMENT;
    }
    const size_t need = loss_workspace(q.tokens);
    if (need && (!workspace || !aligned(workspace, 256))) return SEGTOPK_INVALID_ARGUMENT;
    if (workspace_bytes < 0 || (size_t)workspace_bytes < need) return SEGTOPK_SCRATCH_TOO_SMALL;

    if (!q.tokens) {
        return status(launch(no_rows_kernel, dim3(1), 1, stream, 0, q.loss));
    }
    LossArgs a{};
    a.stride = q.logits.stride;
    a.dstride = q.dlogits.stride;
    a.token_ids = q.token_ids;
    a.old_logp = q.old_logp;
    a.ref_logp = q.ref_logp;
    a.advantages = q.advantages;
    a.logp = q.logp;
    a.loss = q.loss;
    a.term = static_cast<double *>(workspace);
    uint32_t *live = reinterpret_cast<uint32_t *>(a.term + term_bytes(q.tokens) / 8);
    a.live = live;
    a.arrived = live + live_bytes(q.tokens) / 4;
    a.tokens = (uint32_t)q.tokens;
    a.vocab = (uint32_t)q.vocab;
    a.wide = q.id_type == SEGTOPK_KEY_I64;
    a.answers = (double)q.num_segments;
    a.clip_low = q.clip_low;
    a.clip_high = q.clip_high;
    a.kl_coef = q.kl_coef;
    a.temperature = q.temperature;
    a.grad_scale = q.grad_scale;
    // The first part rounded down, so that the rest is positive; both within the
    // normal range, at the temperatures next to zero and infinity too.
    const double factor =
        std::fmin(std::fmax(kLog2e / q.temperature, 2.0 * (double)FLT_MIN), (double)FLT_MAX);
    a.factor = (float)factor;
    if ((double)a.factor >= factor) a.factor = std::nextafter(a.factor, 0.0f);
    a.rest = std::fmax((float)(factor - (double)a.factor), FLT_MIN);
    const int64_t groups = q.num_segments < kCountBlocks ? q.num_segments : kCountBlocks;
    if (launch(count_kernel, dim3(groups ? (unsigned)groups : 1u), kCountThreads, stream, 0,
               q.token_ids, a.wide, a.tokens, a.vocab, q.segment_offsets, (uint32_t)q.num_segments,
               live, a.arrived) != hipSuccess)
        return SEGTOPK_HIP_ERROR;
    return with_type(q.logits.type, [&](auto v) {
        using T = decltype(v);
        const T *in = static_cast<const T *>(q.logits.data);
        T *out = static_cast<T *>(q.dlogits.data);
        const auto go = [&](auto with_grad, auto stream_stores, auto threads) {
            constexpr int kThreads = decltype(threads)::value;
            constexpr bool kGrad = decltype(with_grad)::value;
            constexpr bool kStream = decltype(stream_stores)::value;
            return status(launch(row_kernel<T, kGrad, kStream, kThreads>, dim3(a.tokens), kThreads,
                                 stream, 0, in, out, a));
        };
        const auto by_length = [&](auto with_grad, auto stream_stores) {
            // The smallest workgroup that holds a row in registers.  4096 rows of
            // bf16, by 256, 512 and 1024 threads: 1000 logits 24, 32, 53 us; 8000
            // 32, 37, 58; 16000 53, 45, 63; 32000 105, 88, 78.
            const int64_t bytes = q.vocab * (int64_t)sizeof(T);
            return bytes <= 256 * kAtOnce * 16
                       ? go(with_grad, stream_stores, std::integral_constant<int, 256>{})
                   : bytes <= 512 * kAtOnce * 16
                       ? go(with_grad, stream_stores, std::integral_constant<int, 512>{})
                       : go(with_grad, stream_stores, std::integral_constant<int, 1024>{});
        };
        if (!grad) return by_length(std::false_type{}, std::false_type{});
        return streams(q.tokens * q.vocab * (int64_t)sizeof(T))
                   ? by_length(std::true_type{}, std::true_type{})
                   : by_length(std::true_type{}, std::false_type{});
    });
}
