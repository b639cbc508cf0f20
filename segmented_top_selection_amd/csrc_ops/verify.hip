// verify.hip -- drafted tokens verified against the target's probabilities, and the
// token behind the last that stands.
//
//   p = softmax(target row / temperature),  q = softmax(draft row / temperature)
//   a drafted token t stands if u q(t) < p(t)
//   behind the last that stands: the lowest c whose running sum of w passes
//   v sum(w), with w = max(p - q, 0) at the first that does not stand, and w = p
//   behind all drafts; u and v are the caller's uniform numbers
//
// The running sum passes a border at each of some 10^5 tokens, a few 10^-6 of the
// whole apart: sums of 32 bits, 10^-7 off, would pick another token once in a
// hundred calls.  All is in 64 bits, whose vector rate is that of 32 here: 2^t is
// a polynomial on [-1/2, 1/2] and a shift of the exponent, some 15 instructions for
// an element that takes as long to load.
//
//   stats_kernel  every row in chunks: the maximum, the sum of 2^(x - max) (the
//                 place of the maximum, for temperature 0)
//   pick_kernel   a request in chunks: each workgroup sees from the statistics
//                 which drafts stand, and adds up its chunk of the one row that is
//                 drawn from; the last of a request to arrive finds the token
#include <cmath>
#include <type_traits>

#include "ops_common.h"

namespace segtopk_ops {
namespace {

constexpr double kLog2e = 1.44269504088896340736;
constexpr double kLn2 = 0.693147180559945309417;
constexpr int kMostChunks = 64;  // of a row

struct RowStat {
    double sum;  // of 2^((x - max) factor); NaN: no distribution
    float max;
    uint32_t at;  // temperature 0: the lowest index of the maximum
};

struct VerifyArgs {
    int64_t target_stride, draft_stride;
    const void *tokens_in;
    void *tokens;
    const int64_t *offsets;
    const float *temperatures, *accept, *sample;
    int32_t *counts;
    RowStat *stats;   // [rows][chunks]: the target's rows, then the drafts'
    double *sums;     // [requests][chunks][2]: of w and of p
    uint32_t *arrived;  // [requests]
    double temperature;
    uint32_t drafts, requests, vocab, wide, has_draft;
    uint32_t chunk, chunks;  // elements of a chunk, chunks of a row
};

// 2^t for t <= 0.  The series of 2^f up to f^9: 7e-12 off at most.
__device__ inline double power2(double t) {
    if (t < -1100.0) t = -1100.0;
    const double n = rint(t), f = t - n;
    constexpr double l = kLn2;
    constexpr double c2 = l * l / 2, c3 = c2 * l / 3, c4 = c3 * l / 4, c5 = c4 * l / 5,
                     c6 = c5 * l / 6, c7 = c6 * l / 7, c8 = c7 * l / 8, c9 = c8 * l / 9;
    double p = fma(f, c9, c8);
    p = fma(p, f, c7);
    p = fma(p, f, c6);
    p = fma(p, f, c5);
    p = fma(p, f, c4);
    p = fma(p, f, c3);
    p = fma(p, f, c2);
    p = fma(p, f, l);
    p = fma(p, f, 1.0);
    return ldexp(p, (int)n);
}

__device__ inline float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ inline int64_t draft_offset(const VerifyArgs &a, uint32_t r) {
    const int64_t v = a.offsets[r];
    return v < 0 ? 0 : v > (int64_t)a.drafts ? (int64_t)a.drafts : v;
}

__device__ inline int64_t drafted(const VerifyArgs &a, int64_t i) {
    return a.wide ? static_cast<const int64_t *>(a.tokens_in)[i]
                  : (int64_t) static_cast<const int32_t *>(a.tokens_in)[i];
}
__device__ inline void put(const VerifyArgs &a, int64_t i, int64_t token) {
    if (a.wide) static_cast<int64_t *>(a.tokens)[i] = token;
    else static_cast<int32_t *>(a.tokens)[i] = (int32_t)token;
}

__device__ inline RowStat join(const RowStat &a, const RowStat &b, double factor, bool greedy) {
    RowStat r;
    r.max = a.max > b.max ? a.max : b.max;
    if (greedy) {
        r.sum = a.sum + b.sum;
        r.at = a.max > b.max || (a.max == b.max && a.at < b.at) ? a.at : b.at;
    } else {
        const double m = (double)shift_of(r.max);
        r.sum = a.sum * power2(((double)a.max - m) * factor) + b.sum * power2(((double)b.max - m) * factor);
        r.at = 0;
    }
    return r;
}
__device__ inline RowStat from_lane(const RowStat &s, int d) {
    return {__shfl_xor(s.sum, d), __shfl_xor(s.max, d), __shfl_xor(s.at, d)};
}

// The request of a row of the target, or of a draft.
__device__ inline uint32_t request_of(const VerifyArgs &a, uint32_t row, bool draft) {
    uint32_t lo = 0, hi = a.requests;  // the last request that begins at or before the row
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (draft_offset(a, mid) + (draft ? 0 : mid) <= (int64_t)row) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ inline double temperature_of(const VerifyArgs &a, uint32_t request) {
    return a.temperatures ? (double)a.temperatures[request] : a.temperature;
}

template <class T>
__global__ __launch_bounds__(kOpThreads) void stats_kernel(const T *target, const T *draft,
                                                           VerifyArgs a) {
    using P = Piece<T>;
    constexpr int kAtOnce = 2;
    __shared__ RowStat part[kOpThreads / 64];
    const uint32_t chunk = blockIdx.x % a.chunks, row = blockIdx.x / a.chunks;
    const uint32_t targets = a.drafts + a.requests, i = threadIdx.x;
    if (i == 0 && chunk == 0 && row < a.requests) a.arrived[row] = 0u;
    const bool of_draft = row >= targets;
    const uint32_t r = of_draft ? row - targets : row;
    const double temperature =
        a.temperatures ? temperature_of(a, request_of(a, r, of_draft)) : a.temperature;
    const bool greedy = !(temperature > 0.0);
    if (greedy && of_draft) return;  // not asked for
    const double factor = greedy ? 1.0 : kLog2e / temperature;
    const T *x = of_draft ? draft + (int64_t)r * a.draft_stride : target + (int64_t)r * a.target_stride;
    const uint32_t begin = chunk * a.chunk;
    const uint32_t end = a.vocab - begin < a.chunk ? a.vocab : begin + a.chunk;
    RowStat st{0.0, -INFINITY, UINT32_MAX};
    // Pieces from the chunk's begin on; the elements past them one by one.
    const uint32_t pieces = (end - begin) / P::N;
    const T none = (T)-INFINITY;
    const auto add = [&](const float *v, int n, uint32_t at0, uint32_t step) {
        float m = st.max;
        bool odd = false;
        for (int k = 0; k < n; ++k) {
            if (greedy) {
                if (v[k] > m) st.at = at0 + (uint32_t)(k / P::N) * step + (uint32_t)(k % P::N);
                odd = odd || !(v[k] < INFINITY);
            }
            m = v[k] > m ? v[k] : m;
        }
        if (greedy) {
            if (odd) st.sum = NAN;
        } else {
            const double o = (double)shift_of(m);
            double s = st.sum * power2(((double)st.max - o) * factor);
            for (int k = 0; k < n; ++k) s += power2(((double)v[k] - o) * factor);
            st.sum = s;
        }
        st.max = m;
    };
    for (uint32_t u0 = i; u0 < pieces; u0 += kOpThreads * kAtOnce) {
        float v[kAtOnce * P::N];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const uint32_t u = u0 + j * kOpThreads;
            typename P::vec w = (typename P::vec)none;
            if (u < pieces) w = load_piece(x + begin + (size_t)u * P::N);
            const typename P::f32 f = widen<T>(w);
#pragma unroll
            for (int k = 0; k < P::N; ++k) v[j * P::N + k] = f[k];
        }
        add(v, kAtOnce * P::N, begin + u0 * P::N, kOpThreads * P::N);
    }
    const uint32_t single = begin + pieces * P::N + i;
    if (single < end) {
        const float v[1] = {(float)x[single]};
        add(v, 1, single, 0);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) st = join(st, from_lane(st, d), factor, greedy);
    if (i % 64 == 0) part[i / 64] = st;
    __syncthreads();
    if (i) return;
    for (int w = 1; w < kOpThreads / 64; ++w) st = join(st, part[w], factor, greedy);
    a.stats[(int64_t)row * a.chunks + chunk] = st;
}

// A row's statistics from those of its chunks.
__device__ inline RowStat row_stat(const VerifyArgs &a, int64_t row, double factor, bool greedy) {
    const RowStat *s = a.stats + row * a.chunks;
    RowStat st = s[0];
    for (uint32_t c = 1; c < a.chunks; ++c) st = join(st, s[c], factor, greedy);
    return st;
}
// Some logit is above -inf, and none is NaN or +inf.
__device__ inline bool good(const RowStat &s) { return s.max > -INFINITY && s.sum == s.sum; }

// What a request's token is drawn from.
struct Source {
    double max, inverse, draft_max, draft_inverse;  // of the rows
    int64_t row, draft;  // draft -1: none
    int64_t certain;     // the token that was certain and does not stand, or -1
};

template <class T>
__global__ __launch_bounds__(kOpThreads) void pick_kernel(const T *target, const T *draft,
                                                          VerifyArgs a) {
    using P = Piece<T>;
    __shared__ uint32_t stop, arrival, chosen;
    __shared__ Source src;
    __shared__ double scan[kOpThreads];
    __shared__ double base, goal;
    __shared__ uint32_t plain;
    const uint32_t chunk = blockIdx.x % a.chunks, r = blockIdx.x / a.chunks, i = threadIdx.x;
    const int64_t first = draft_offset(a, r);
    const int64_t after = draft_offset(a, r + 1);
    const uint32_t n = after > first ? (uint32_t)(after - first) : 0u;
    const int64_t row0 = first + r;
    const double temperature = temperature_of(a, r);
    const bool greedy = !(temperature > 0.0);
    const double factor = greedy ? 1.0 : kLog2e / temperature;
    const int64_t targets = (int64_t)a.drafts + a.requests;
    const bool certain = greedy || !a.has_draft;

    if (i == 0) stop = n;
    __syncthreads();
    for (uint32_t j0 = 0; j0 < n && stop == n; j0 += kOpThreads) {
        const uint32_t j = j0 + i;
        bool stands = true;
        if (j < n) {
            const int64_t t = drafted(a, first + j);
            const RowStat s = row_stat(a, row0 + j, factor, greedy);
            stands = t >= 0 && t < (int64_t)a.vocab && good(s);
            if (stands && greedy) {
                stands = t == (int64_t)s.at;
            } else if (stands) {
                const double x = (double)(float)target[(row0 + j) * a.target_stride + t];
                const double p = power2((x - (double)s.max) * factor) / s.sum;
                double q = 1.0;
                if (!certain) {
                    const RowStat d = row_stat(a, targets + first + j, factor, false);
                    const double y = (double)(float)draft[(first + j) * a.draft_stride + t];
                    q = power2((y - (double)d.max) * factor) / d.sum;
                    stands = good(d);
                }
                stands = stands && (double)a.accept[first + j] * q < p;
            }
        }
        __syncthreads();  // everyone has looked at `stop`
        if (!stands) atomicMin(&stop, j);
        __syncthreads();
    }
    const uint32_t stood = stop;
    if (i == 0) {
        const RowStat s = row_stat(a, row0 + stood, factor, greedy);
        src.row = row0 + stood;
        src.max = (double)s.max;
        src.inverse = good(s) ? 1.0 / s.sum : NAN;
        src.draft = src.certain = -1;
        if (stood < n) {
            if (certain) {
                src.certain = drafted(a, first + stood);
            } else {
                src.draft = first + stood;
                const RowStat d = row_stat(a, targets + first + stood, factor, false);
                src.draft_max = (double)d.max;
                src.draft_inverse = 1.0 / d.sum;
                if (!good(d)) src.inverse = NAN;
            }
        }
        if (greedy) chosen = s.at;
    }
    __syncthreads();
    const bool none = src.inverse != src.inverse;
    if (chunk == 0) {
        for (uint32_t j = i; j <= n; j += kOpThreads)
            if (j < stood) put(a, row0 + j, drafted(a, first + j));
            else if (j > stood || none) put(a, row0 + j, -1);
            else if (greedy) put(a, row0 + j, chosen);
        if (i == 0) a.counts[r] = (int32_t)(stood + (none ? 0u : 1u));
    }
    if (greedy || none) return;

    const T *x = target + src.row * a.target_stride;
    const T *y = src.draft >= 0 ? draft + src.draft * a.draft_stride : nullptr;
    const auto probability = [&](float v) { return power2(((double)v - src.max) * factor) * src.inverse; };
    const auto weight = [&](double p, float v, uint32_t c) {
        if (y) p -= power2(((double)v - src.draft_max) * factor) * src.draft_inverse;
        else if ((int64_t)c == src.certain) p = 0.0;
        return p > 0.0 ? p : 0.0;
    };
    {
        const uint32_t begin = chunk * a.chunk;
        const uint32_t end = a.vocab - begin < a.chunk ? a.vocab : begin + a.chunk;
        const uint32_t pieces = (end - begin) / P::N;
        double w = 0.0, p = 0.0;
        for (uint32_t u = i; u < pieces; u += kOpThreads) {
            const uint32_t at = begin + u * P::N;
            const typename P::f32 f = widen<T>(load_piece(x + at));
            typename P::f32 g = f;
            if (y) g = widen<T>(load_piece(y + at));
#pragma unroll
            for (int k = 0; k < P::N; ++k) {
                const double one = probability(f[k]);
                p += one;
                w += weight(one, g[k], at + k);
            }
        }
        const uint32_t single = begin + pieces * P::N + i;
        if (single < end) {
            const double one = probability((float)x[single]);
            p += one;
            w += weight(one, y ? (float)y[single] : 0.0f, single);
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            w += __shfl_xor(w, d);
            p += __shfl_xor(p, d);
        }
        if (i % 64 == 0) {
            scan[i / 64] = w;
            scan[4 + i / 64] = p;
        }
        __syncthreads();
        if (i == 0) {
            for (int k = 1; k < kOpThreads / 64; ++k) {
                w += scan[k];
                p += scan[4 + k];
            }
            double *s = a.sums + ((int64_t)r * a.chunks + chunk) * 2;
            __hip_atomic_store(s, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(s + 1, p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // Both are past this XCD's cache before the chunk counts as done.
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            arrival = __hip_atomic_fetch_add(&a.arrived[r], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __syncthreads();
    if (arrival + 1u != a.chunks) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    if (i == 0) {
        const double *s = a.sums + (int64_t)r * a.chunks * 2;
        const auto sum_of = [&](uint32_t c, uint32_t which) {
            return __hip_atomic_load(s + c * 2 + which, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        };
        double total = 0.0;
        for (uint32_t c = 0; c < a.chunks; ++c) total += sum_of(c, 0);
        plain = total > 0.0 ? 0u : 1u;  // p is nowhere above q: p itself
        if (plain)
            for (uint32_t c = 0; c < a.chunks; ++c) total += sum_of(c, 1);
        goal = (double)a.sample[r] * total;
        // The first chunk that passes the goal, or the last with anything in it.
        double before = 0.0;
        chosen = 0;
        base = 0.0;
        for (uint32_t c = 0; c < a.chunks; ++c) {
            const double v = sum_of(c, plain);
            if (v > 0.0) {
                chosen = c;
                base = before;
            }
            before += v;
            if (before > goal) break;
        }
    }
    __syncthreads();
    const uint32_t begin = chosen * a.chunk;
    const uint32_t end = a.vocab - begin < a.chunk ? a.vocab : begin + a.chunk;
    const uint32_t each = (end - begin + kOpThreads - 1) / kOpThreads;
    const uint32_t b = begin + i * each < end ? begin + i * each : end;
    const uint32_t e = b + each < end ? b + each : end;
    const auto weight_at = [&](uint32_t c) {
        const double p = probability((float)x[c]);
        return plain ? p : weight(p, y ? (float)y[c] : 0.0f, c);
    };
    double mine = 0.0;
    for (uint32_t c = b; c < e; ++c) mine += weight_at(c);
    scan[i] = mine;
    __syncthreads();
    double before = base;
    for (uint32_t k = 0; k < i; ++k) before += scan[k];
    __syncthreads();
    if (i == 0) chosen = UINT32_MAX;
    __syncthreads();
    if (before + mine > goal) {  // here, or in a thread before
        for (uint32_t c = b; c < e; ++c) {
            const double w = weight_at(c);
            before += w;
            if (w > 0.0 && before > goal) {
                atomicMin(&chosen, c);
                break;
            }
        }
    }
    __syncthreads();
    if (chosen == UINT32_MAX) {
        // Rounding alone keeps the goal out of reach: the last of any weight.
        __syncthreads();
        if (i == 0) arrival = 0;
        __syncthreads();
        for (uint32_t c = e; c-- > b;)
            if (weight_at(c) > 0.0) {
                atomicMax(&arrival, c);
                break;
            }
        __syncthreads();
        if (i == 0) chosen = arrival;
    }
    if (i == 0) put(a, src.row, chosen);
}

struct Cut {
    uint32_t chunk, chunks;
};

// Chunks of 16384 elements, or less where there are few rows: a quarter is what a
// workgroup takes at one go.
Cut cut_of(int64_t drafts, int64_t requests, int64_t vocab) {
    const int64_t rows = 2 * drafts + requests;
    int64_t chunk = 16384;
    while (chunk > 4096 && rows * ((vocab + chunk - 1) / chunk) < 1024) chunk /= 2;
    const int64_t least = (vocab + kMostChunks - 1) / kMostChunks;
    if (chunk < least) chunk = (least + 4095) / 4096 * 4096;
    return {(uint32_t)chunk, (uint32_t)((vocab + chunk - 1) / chunk)};
}

bool good_verify_sizes(int64_t drafts, int64_t requests, int64_t vocab) {
    return drafts >= 0 && requests >= 0 && drafts < (1 << 22) && requests < (1 << 22) &&
           drafts + requests < (1 << 22) && vocab >= 1 && vocab <= INT32_MAX;
}

struct VerifySpace {
    int64_t stats, sums, arrived, bytes;
};
VerifySpace verify_space(int64_t drafts, int64_t requests, const Cut &c) {
    VerifySpace s;
    s.stats = 0;
    s.sums = s.stats + (2 * drafts + requests) * c.chunks * (int64_t)sizeof(RowStat);
    s.arrived = s.sums + requests * c.chunks * 16;
    s.bytes = s.arrived + requests * 4;
    return s;
}

}  // namespace
}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int64_t segtopk_verify_workspace(int64_t num_drafts, int64_t num_requests,
                                            int64_t vocab) {
    if (!good_verify_sizes(num_drafts, num_requests, vocab) || !num_requests) return 0;
    return verify_space(num_drafts, num_requests, cut_of(num_drafts, num_requests, vocab)).bytes;
}

extern "C" int segtopk_verify_drafts(const segtopk_verify_args *args, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream) {
    if (!args) return SEGTOPK_INVALID_ARGUMENT;
    const segtopk_verify_args &q = *args;
    if (!good_verify_sizes(q.num_drafts, q.num_requests, q.vocab) || !index_bytes(q.id_type) ||
        !std::isfinite(q.temperature) || q.temperature < 0.0)
        return SEGTOPK_INVALID_ARGUMENT;
    if (!q.num_requests) return q.num_drafts ? SEGTOPK_INVALID_ARGUMENT : SEGTOPK_OK;
    const int ib = index_bytes(q.id_type);
    const auto floats = [](const float *p) { return p && aligned(p, 4); };
    if (!good_rows(&q.target, q.vocab) || !q.draft_offsets || !aligned(q.draft_offsets, 8) ||
        !q.tokens || !aligned(q.tokens, ib) || !floats(q.sample) || !q.counts ||
        !aligned(q.counts, 4) || (q.temperatures && !aligned(q.temperatures, 4)))
        return SEGTOPK_INVALID_ARGUMENT;
    if (q.num_drafts && (!q.draft_tokens || !aligned(q.draft_tokens, ib) || !floats(q.accept)))
        return SEGTOPK_INVALID_ARGUMENT;
    const bool has_draft = q.num_drafts && q.draft.data;
    if (has_draft && (!good_rows(&q.draft, q.vocab) || q.draft.type != q.target.type))
        return SEGTOPK_INVALID_ARGUMENT;
    const Cut cut = cut_of(q.num_drafts, q.num_requests, q.vocab);
    if ((2 * q.num_drafts + q.num_requests) * cut.chunks > kMostBlocks) return SEGTOPK_NOT_SUPPORTED;
    const VerifySpace s = verify_space(q.num_drafts, q.num_requests, cut);
    if (workspace_bytes < s.bytes) return SEGTOPK_SCRATCH_TOO_SMALL;
    if (!workspace || !aligned(workspace, 256)) return SEGTOPK_INVALID_ARGUMENT;
    char *ws = static_cast<char *>(workspace);
    VerifyArgs a{};
    a.target_stride = q.target.stride;
    a.draft_stride = q.draft.stride;
    a.tokens_in = q.draft_tokens;
    a.tokens = q.tokens;
    a.offsets = q.draft_offsets;
    a.temperatures = q.temperatures;
    a.accept = q.accept;
    a.sample = q.sample;
    a.counts = q.counts;
    a.stats = reinterpret_cast<RowStat *>(ws + s.stats);
    a.sums = reinterpret_cast<double *>(ws + s.sums);
    a.arrived = reinterpret_cast<uint32_t *>(ws + s.arrived);
    a.temperature = q.temperature;
    a.drafts = (uint32_t)q.num_drafts;
    a.requests = (uint32_t)q.num_requests;
    a.vocab = (uint32_t)q.vocab;
    a.wide = q.id_type == SEGTOPK_KEY_I64;
    a.has_draft = has_draft;
    a.chunk = cut.chunk;
    a.chunks = cut.chunks;
    const unsigned rows = a.drafts + a.requests + (has_draft ? a.drafts : 0u);
    return with_type(q.target.type, [&](auto v) -> int {
        using T = decltype(v);
        const T *target = static_cast<const T *>(q.target.data);
        const T *draft = has_draft ? static_cast<const T *>(q.draft.data) : nullptr;
        if (launch(stats_kernel<T>, dim3(rows * a.chunks), kOpThreads, stream, 0, target, draft,
                   a) != hipSuccess)
            return SEGTOPK_HIP_ERROR;
        return status(launch(pick_kernel<T>, dim3(a.requests * a.chunks), kOpThreads, stream, 0,
                             target, draft, a));
    });
}
