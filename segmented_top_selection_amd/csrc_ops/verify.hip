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
// one of 32 roots in LDS, a polynomial of degree 4 on [-1/64, 1/64], 8e-14 off, and
// an addition to the exponent, some 14 instructions for an element that takes as long
// to load.  (Without roots it is a polynomial of degree 9.)
//
//   stats_kernel  every row in chunks: the maximum, the sum of 2^(x - max) (the
//                 place of the maximum, for temperature 0)
//   pick_kernel   a request in chunks: each workgroup sees from the statistics
//                 which drafts stand, and adds up its chunk of the one row that is
//                 drawn from; the last of a request to arrive finds the token
//
// 64 requests of up to seven drafts over 131072 entries in bf16: 75 us, of which 45 are the
// statistics (27 without the powers; without roots, by a polynomial of degree 7, 48, and then 38
// without the loads) and 31 the pick.  One request of 32003: 12.4 us, two launches and the pick's chain of
// offsets, drafts, statistics, parts and places.
#include <cmath>
#include <type_traits>

#include "ops_common.h"

namespace segtopk_ops {
namespace {

constexpr double kLog2e = 1.44269504088896340736;
constexpr uint32_t kMostChunks = 16;   // of a row for its statistics, one to a lane of 16
constexpr uint32_t kMostParts = 256;   // of the row that is drawn from, one to a thread
constexpr uint32_t kPart = kOpThreads * 4;  // the least of its parts

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
    double *sums;     // [requests][parts][waves][2]: of w and of p
    uint32_t *arrived;  // [requests]
    double temperature;
    uint32_t drafts, requests, vocab, wide, has_draft;
    uint32_t chunk, chunks;  // elements of a chunk, chunks of a row
    uint32_t part, parts;    // the same of the row that is drawn from
};

// 2^(j / 32).
__device__ const double kRoots[32] = {
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0};
// They in LDS as words: the high one without j << 15, see power().  32 of 8 bytes are all the
// banks once, so that lanes meet only where they read the same.
struct Roots {
    uint2 of[32];
};
__device__ inline void fill(Roots &roots) {
    const uint32_t j = threadIdx.x;
    if (j < 32) {
        const double v = kRoots[j];
        roots.of[j] = uint2{(uint32_t)__double2loint(v), (uint32_t)__double2hiint(v) - (j << 15)};
    }
}

// 2^(x factor - shift), `shift` being max factor to the nearest integer, for x <= max.  What is
// below 2^-1000, -inf too, gives that.
struct Power {
    double factor, round, low;  // 1.5 * 2^47 - shift, and the x of 2^-1000
};
__device__ inline double shift_of(float max, double factor) {
    return max == -INFINITY ? 0.0 : rint((double)max * factor);
}
// Past 2^40 the product leaves no 32nds of a whole number.  Two logits are 2^-24 of the larger
// apart at least, so that all others than the largest are nothing there, and are with the factor
// that makes the product 2^40 too.
// `span` is 1000 / factor.
__device__ inline Power power_of(float max, double factor, double span) {
    if (fabs((double)max * factor) > 0x1p40 && max != -INFINITY) {
        factor = 0x1p40 / fabs((double)max);
        span = 1000.0 / factor;
    }
    return {factor, 0x1.8p47 - shift_of(max, factor), (max == -INFINITY ? 0.0 : (double)max) - span};
}
// log2(e) / temperature; from 2^830 on any two logits are as far apart as can be, and products
// with a logit stay finite.
__device__ inline double factor_of(double temperature) {
    return fmin(kLog2e / temperature, 0x1p830);
}
// What a sum by one maximum is multiplied by to become one by a larger: a power of two.
// (A sum by -inf is n 2^-1000 for n elements, and what it is multiplied by is never above one:
// beside a row's sum, of which the largest element alone is 2^-0.5 or more, it is nothing.)
__device__ inline double between(float from, float to, double factor) {
    const double d = shift_of(from, factor) - shift_of(to, factor);
    const int e = d > 0.0 ? 0 : d < -1020.0 ? -1020 : (int)d;
    return __hiloint2double((1023 + e) << 20, 0);
}
// Its exponent is n + j / 32 + f: an addition that leaves 32nds the last bit has n and j in the
// low word, f is what is over, and 2^f the polynomial of degree 4 that goes through it at the
// Chebyshev points of [-1/64, 1/64], 8e-14 off: as near as a running sum of 10^5 numbers in 64
// bits is.  (Degree 3, 7e-11 off: 64 requests 73.8 against 74.7 us.)  The whole low word goes 15
// bits up to the root's high word, n into the exponent, and takes back j << 15.
struct Factors {
    double root, poly;  // their product is the power
};
__device__ inline Factors factors(const Power &a, double x, const Roots &roots) {
    const double s = fma(x, a.factor, a.round), f = fma(x, a.factor, a.round - s);
    const uint32_t k = (uint32_t)__double2loint(s);
    const uint2 r = roots.of[k % 32];
    double p = fma(f, 0.009618176115571158, 0.055504515573860415);
    p = fma(p, f, 0.24022650695623157);
    p = fma(p, f, 0.6931471805351095);
    p = fma(p, f, 1.0);
    return {__hiloint2double((int)(r.y + (k << 15)), (int)r.x), p};
}
// The sum so far and one power more.
__device__ inline double add_power(const Power &a, float v, const Roots &roots, double sum) {
    const Factors p = factors(a, fmax((double)v, a.low), roots);
    return fma(p.root, p.poly, sum);
}
// A power, where what is ruled out, or as good as that, has to be nothing.
__device__ inline double power_or_zero(const Power &a, float v, const Roots &roots) {
    const double x = fmax((double)v, a.low);
    const Factors p = factors(a, x, roots);
    return x <= a.low ? 0.0 : p.root * p.poly;
}

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

template <int L> __device__ inline float largest(float v) {
    return join<L>(v, [](float a, float b) { return a > b ? a : b; });
}
template <int L> __device__ inline uint32_t lowest(uint32_t v) {
    return join<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L> __device__ inline double total_of(double v) {
    return join<L>(v, [](double a, double b) { return a + b; });
}

// The statistics of L lanes as one.
template <int L> __device__ inline RowStat join_lanes(const RowStat &s, double factor, bool greedy) {
    const float m = largest<L>(s.max);
    if (greedy) return {total_of<L>(s.sum), m, lowest<L>(s.max == m ? s.at : UINT32_MAX)};
    return {total_of<L>(s.sum * between(s.max, m, factor)), m, 0u};
}

template <class T, int AT_ONCE>
__global__ __launch_bounds__(kOpThreads) void stats_kernel(const T *target, const T *draft,
                                                           VerifyArgs a) {
    using P = Piece<T>;
    constexpr int kAtOnce = AT_ONCE, kElements = kAtOnce * P::N;
    __shared__ RowStat part[kOpThreads / 64];
    __shared__ Roots roots;
    fill(roots);
    const uint32_t chunk = blockIdx.x % a.chunks, row = blockIdx.x / a.chunks;
    const uint32_t targets = a.drafts + a.requests, i = threadIdx.x;
    if (i == 0 && chunk == 0 && row < a.requests) a.arrived[row] = 0u;
    const bool of_draft = row >= targets;
    const uint32_t r = of_draft ? row - targets : row;
    const double temperature =
        a.temperatures ? temperature_of(a, request_of(a, r, of_draft)) : a.temperature;
    const bool greedy = !(temperature > 0.0);
    if (greedy && of_draft) return;  // not asked for
    const double factor = greedy ? 1.0 : factor_of(temperature), span = 1000.0 / factor;
    const T *x = of_draft ? draft + (int64_t)r * a.draft_stride : target + (int64_t)r * a.target_stride;
    const uint32_t begin = chunk * a.chunk;
    const uint32_t end = a.vocab - begin < a.chunk ? a.vocab : begin + a.chunk;
    // Pieces from the chunk's begin on; the elements past them one by one.
    const uint32_t pieces = (end - begin) / P::N;
    const T none = (T)-INFINITY;
    RowStat st{0.0, -INFINITY, UINT32_MAX};  // of the thread
    bool odd = false;
    const auto add = [&](const float *v, uint32_t at0) {
        float m = st.max;
        if (greedy) {
#pragma unroll
            for (int k = 0; k < kElements; ++k) {
                odd = odd || !(v[k] < INFINITY);
                if (v[k] > m) {
                    st.at = at0 + (uint32_t)(k / P::N) * kOpThreads * P::N + k % P::N;
                    m = v[k];
                }
            }
        } else {
            // This maximum keeps NaN.
#pragma unroll
            for (int k = 0; k < kElements; k += 2)
                m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, v[k]), v[k + 1]);
            odd = odd || !(m < INFINITY);
            const Power e = power_of(m, factor, span);
            double s = st.sum * between(st.max, m, factor);
#pragma unroll
            for (int k = 0; k < kElements; ++k) s = add_power(e, v[k], roots, s);
            st.sum = s;
        }
        st.max = m;
    };
    // The last turn is theirs, if there are any: the same code, which comes into the cache as it is
    // needed.
    const uint32_t whole = (pieces + kOpThreads * kAtOnce - 1) / (kOpThreads * kAtOnce);
    const uint32_t turns = whole + (begin + pieces * P::N < end ? 1u : 0u);
#pragma unroll 1
    for (uint32_t turn = 0; turn < turns; ++turn) {
        const uint32_t u0 = turn * kOpThreads * kAtOnce + i, single = begin + pieces * P::N + i;
        float v[kElements];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const uint32_t u = u0 + j * kOpThreads;
            typename P::vec w = (typename P::vec)none;
            if (u < pieces) w = load_piece(x + begin + (size_t)u * P::N);
            const typename P::f32 f = widen<T>(w);
#pragma unroll
            for (int k = 0; k < P::N; ++k) v[j * P::N + k] = f[k];
        }
        if (turn == whole && single < end) v[0] = (float)x[single];
        if (!turn) __syncthreads();  // the roots are there, behind the first loads
        add(v, turn == whole ? single : begin + u0 * P::N);
    }
    if (odd) st.sum = NAN;
    st = join_lanes<64>(st, factor, greedy);
    if (i % 64 == 0) part[i / 64] = st;
    __syncthreads();
    if (i >= 16) return;
    if (i < kOpThreads / 64) st = part[i];
    else st = {0.0, -INFINITY, UINT32_MAX};
    st = join_lanes<16>(st, factor, greedy);
    if (i == 0) a.stats[(int64_t)row * a.chunks + chunk] = st;
}

// A row's statistics from those of its chunks, by 16 lanes.
__device__ inline RowStat row_stat(const VerifyArgs &a, int64_t row, double factor, bool greedy) {
    const uint32_t lane = threadIdx.x % 16;
    RowStat s{0.0, -INFINITY, UINT32_MAX};
    if (lane < a.chunks) s = a.stats[row * a.chunks + lane];
    return join_lanes<16>(s, factor, greedy);
}
// Some logit is above -inf, and none is NaN or +inf.
__device__ inline bool good(const RowStat &s) { return s.max > -INFINITY && s.sum == s.sum; }

// What a request's token is drawn from.
struct Source {
    Power power, draft_power;
    double inverse, draft_inverse;  // of the rows' sums
    int64_t row, draft;  // draft -1: none
    int64_t certain;     // the token that was certain and does not stand, or -1
    uint32_t at;         // temperature 0: the token
};

// v of the lanes that come before by the DPP step, nothing for the others.
template <int STEP, int ROWS> __device__ inline double from_before(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), STEP, ROWS, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), STEP, ROWS, 0xF, false);
    return __hiloint2double(hi, lo);
}
// The sum of all threads' numbers before each, and of all.
struct Scan {
    double before, all;
};
// The sum of the wave's numbers up to each lane's.
__device__ inline double scan_wave(double s) {
    s += from_before<0x111, 0xF>(s);  // 1, 2, 4, 8 lanes before, within rows of 16
    s += from_before<0x112, 0xF>(s);
    s += from_before<0x114, 0xF>(s);
    s += from_before<0x118, 0xF>(s);
    s += from_before<0x142, 0xA>(s);  // the last of the row before, to rows 1 and 3
    s += from_before<0x143, 0xC>(s);  // lane 31, to rows 2 and 3
    return s;
}
__device__ inline Scan scan_threads(double v, double *part) {
    const uint32_t i = threadIdx.x, lane = i % 64;
    const double s = scan_wave(v);
    __syncthreads();  // the last call's numbers have been read
    if (lane == 63) part[i / 64] = s;
    __syncthreads();
    Scan r{s - v, 0.0};
#pragma unroll
    for (uint32_t w = 0; w < kOpThreads / 64; ++w) {
        if (w < i / 64) r.before += part[w];
        r.all += part[w];
    }
    return r;
}

// The first thread whose sum is over the goal; where rounding alone keeps it out of reach, the
// last with anything to add.  `found` was last read before a barrier.
__device__ inline uint32_t find_thread(bool over, bool any, uint32_t *found) {
    const uint64_t o = __ballot(over), n = __ballot(any);
    constexpr uint32_t kOver = 1u << 16, kAny = 1u << 17;
    if (threadIdx.x % 64 == 0)
        found[threadIdx.x / 64] = o   ? kOver + threadIdx.x + (uint32_t)__builtin_ctzll(o)
                                  : n ? kAny + threadIdx.x + 63u - (uint32_t)__builtin_clzll(n)
                                      : 0u;
    __syncthreads();
    uint32_t at = 0;
#pragma unroll
    for (uint32_t w = 0; w < kOpThreads / 64; ++w)
        if (found[w] && !(at & kOver)) at = found[w];
    return at & (kOver - 1);
}

template <class T>
__global__ __launch_bounds__(kOpThreads) void pick_kernel(const T *target, const T *draft,
                                                          VerifyArgs a) {
    using P = Piece<T>;
    constexpr uint32_t kAtOnce = kOpThreads / 32;  // drafts
    __shared__ uint32_t stop, arrival, found[kOpThreads / 64];
    __shared__ Source src;
    __shared__ RowStat seen[kAtOnce][2];
    __shared__ double likely[kAtOnce][2];
    __shared__ double scan[kOpThreads / 64];
    __shared__ Roots roots;
    fill(roots);
    const uint32_t part = blockIdx.x % a.parts, r = blockIdx.x / a.parts, i = threadIdx.x;
    const int64_t first = draft_offset(a, r);
    const int64_t after = draft_offset(a, r + 1);
    const uint32_t n = after > first ? (uint32_t)(after - first) : 0u;
    const int64_t row0 = first + r;
    const double temperature = temperature_of(a, r);
    const bool greedy = !(temperature > 0.0);
    const double factor = greedy ? 1.0 : factor_of(temperature);
    const int64_t targets = (int64_t)a.drafts + a.requests;
    const bool certain = greedy || !a.has_draft;

    // 16 lanes a row, the target's and the draft's of several drafts at once, until one does
    // not stand; behind the last draft, its row.
    const uint32_t local = i / 32, of_draft = i / 16 % 2;
    for (uint32_t j0 = 0;; j0 += kAtOnce) {
        const uint32_t j = j0 + local;
        if (i == 0) stop = n;
        const bool asked = j <= n && (!of_draft || (j < n && !certain));
        RowStat s{0.0, -INFINITY, 0u};
        int64_t t = -1;
        if (asked) {
            s = row_stat(a, of_draft ? targets + first + j : row0 + j, factor, greedy);
            if (j < n) t = drafted(a, first + j);
        }
        const bool inside = t >= 0 && t < (int64_t)a.vocab;
        __syncthreads();  // the roots are there
        if (i % 16 == 0) {
            double p = of_draft ? 1.0 : 0.0;  // of a draft that was certain
            if (asked && inside && greedy) {
                p = t == (int64_t)s.at ? 1.0 : 0.0;
            } else if (asked && inside) {
                const T v = of_draft ? draft[(first + j) * a.draft_stride + t]
                                     : target[(row0 + j) * a.target_stride + t];
                p = power_or_zero(power_of(s.max, factor, 1000.0 / factor), (float)v, roots) / s.sum;
            }
            seen[local][of_draft] = s;
            likely[local][of_draft] = p;
        }
        __syncthreads();
        if (i % 32 == 0 && j < n) {
            const bool known = good(seen[local][0]) && (certain || good(seen[local][1]));
            if (!(known && inside && (double)a.accept[first + j] * likely[local][1] < likely[local][0]))
                atomicMin(&stop, j);
        }
        __syncthreads();
        const uint32_t here = stop;
        if (here < j0 + kAtOnce) {  // it has been looked at: a draft, or the row behind all
            if (i == 0) {
                const RowStat of_row = seen[here - j0][0], of_q = seen[here - j0][1];
                src.row = row0 + here;
                src.power = power_of(of_row.max, factor, 1000.0 / factor);
                src.inverse = good(of_row) ? 1.0 / of_row.sum : NAN;
                src.draft = src.certain = -1;
                src.at = of_row.at;
                if (here < n && certain) {
                    src.certain = drafted(a, first + here);
                } else if (here < n) {
                    src.draft = first + here;
                    src.draft_power = power_of(of_q.max, factor, 1000.0 / factor);
                    src.draft_inverse = 1.0 / of_q.sum;
                    if (!good(of_q)) src.inverse = NAN;
                }
            }
            break;
        }
    }
    __syncthreads();
    const uint32_t stood = (uint32_t)(src.row - row0);
    const Source from = src;
    const bool none = from.inverse != from.inverse;
    if (part == 0) {
        for (uint32_t j = i; j <= n; j += kOpThreads)
            if (j < stood) put(a, row0 + j, drafted(a, first + j));
            else if (j > stood || none) put(a, row0 + j, -1);
            else if (greedy) put(a, row0 + j, from.at);
        if (i == 0) a.counts[r] = (int32_t)(stood + (none ? 0u : 1u));
    }
    if (greedy || none) return;

    const T *x = target + from.row * a.target_stride;
    const T *y = from.draft >= 0 ? draft + from.draft * a.draft_stride : nullptr;
    const auto probability = [&](float v) {
        return power_or_zero(from.power, v, roots) * from.inverse;
    };
    const auto weight = [&](double p, float v, uint32_t c) {
        if (y) p -= power_or_zero(from.draft_power, v, roots) * from.draft_inverse;
        else if ((int64_t)c == from.certain) p = 0.0;
        return p > 0.0 ? p : 0.0;
    };
    // What is added up of element c.
    struct Both {
        double w, p;
    };
    const auto both = [&](uint32_t c, float v, float g) {
        const double p = probability(v);
        return Both{weight(p, g, c), p};
    };
    // The same code for the workgroup's own part and, by the last to arrive, for what one wave
    // had of the part that the token is in, and for one thread's run of that: code that comes
    // into the cache as it is needed costs more time than the elements.  A thread has a run of
    // elements, four at a time.
    constexpr uint32_t kWaves = kOpThreads / 64;
    uint32_t each = a.part / kOpThreads, begin = part * a.part, end = a.vocab;
    bool plain = false;
    double base = 0.0, goal = 0.0;
    typedef T four __attribute__((ext_vector_type(4), aligned(sizeof(T))));
#pragma unroll 1
    for (uint32_t pass = 0;; ++pass) {
        const uint32_t run = begin + i * each, run_end = run + each < end ? run + each : end;
        const auto read = [&](uint32_t c, four &one, four &two) {
            one = two = (four)(T)-INFINITY;
            if (c + 4 <= run_end) {
                one = *reinterpret_cast<const four *>(x + c);
                if (y) two = *reinterpret_cast<const four *>(y + c);
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (c + k < run_end) {
                        one[k] = x[c + k];
                        if (y) two[k] = y[c + k];
                    }
            }
        };
        Both sum{0.0, 0.0};
        four one, two;
        read(run, one, two);
#pragma unroll 1
        for (uint32_t c = run; c < run_end; c += 4) {
            four next_one, next_two;
            read(c + 4, next_one, next_two);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const Both e = both(c + k, (float)one[k], (float)two[k]);
                sum.w += e.w;
                sum.p += e.p;
            }
            one = next_one;
            two = next_two;
        }
        if (pass) {
            const double m = plain ? sum.p : sum.w;
            const Scan s = scan_threads(m, scan);
            const uint32_t owner =
                find_thread(m > 0.0 && base + s.before + m > goal, m > 0.0, found);
            if (each == 1) {
                if (i == owner) put(a, from.row, run);
                return;
            }
            __syncthreads();
            if (i == owner) scan[0] = base + s.before;
            __syncthreads();
            base = scan[0];
            begin += owner * each;
            end = begin + each < end ? begin + each : end;
            each = (each + kOpThreads - 1) / kOpThreads;
            continue;
        }
        sum.w = total_of<64>(sum.w);
        sum.p = total_of<64>(sum.p);
        if (i % 64 == 0) {
            double *s = a.sums + (((int64_t)r * a.parts + part) * kWaves + i / 64) * 2;
            __hip_atomic_store(s, sum.w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(s + 1, sum.p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // All are past this XCD's cache before the part counts as done.
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        __syncthreads();
        if (i == 0)
            arrival = __hip_atomic_fetch_add(&a.arrived[r], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (arrival + 1u != a.parts) return;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        double w[kWaves], p[kWaves], w_all = 0.0, p_all = 0.0;  // of part i
#pragma unroll
        for (uint32_t k = 0; k < kWaves; ++k) {
            w[k] = p[k] = 0.0;
            if (i < a.parts) {
                const double *s = a.sums + (((int64_t)r * a.parts + i) * kWaves + k) * 2;
                w[k] = __hip_atomic_load(s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                p[k] = __hip_atomic_load(s + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            w_all += w[k];
            p_all += p[k];
        }
        Scan sums = scan_threads(w_all, scan);
        plain = !(sums.all > 0.0);  // p is nowhere above q: p itself
        if (plain) {
            sums = scan_threads(p_all, scan);
            w_all = p_all;
        }
        goal = (double)a.sample[r] * sums.all;
        const uint32_t which =
            find_thread(w_all > 0.0 && sums.before + w_all > goal, w_all > 0.0, found);
        __syncthreads();
        if (i == which) {  // the same among its waves
            double before = sums.before;
            uint32_t wave = 0;
            bool over = false;
#pragma unroll
            for (uint32_t k = 0; k < kWaves; ++k) {
                const double e = plain ? p[k] : w[k];
                if (e > 0.0 && !over) {
                    wave = k;
                    scan[0] = before;
                    over = before + e > goal;
                }
                before += e;
            }
            stop = wave;
        }
        __syncthreads();
        base = scan[0];
        begin = which * a.part + stop * 64 * each;
        end = begin + 64 * each < end ? begin + 64 * each : end;
        each /= kWaves;  // a part is some 1024 elements
    }
}

struct Cut {
    uint32_t chunk, chunks, part, parts;
};

// Chunks of 65536 elements, or less where there are few rows.  By 2048, 4096, 8192 workgroups, new
// inputs in turn: 64 requests of 131072 entries and up to 7 drafts 78, 74, 80 us, 128 and up to 3
// 95, 91, 97, 1024 of 32000 and one 188, 184, 187; but 32 of 131072 45, 48, 50, 48 of 100000 52, 57,
// 57, 64 of 65536 51, 54, 56, 64 of 128256 and up to 5 65, 70: neither of the first two is ahead
// everywhere.
// Parts of 1024 elements, or up to 8192 where there are many requests, since each workgroup finds
// out for itself where the drafts stop.  By 512 and 1024 workgroups before they grow: 8 requests
// of 131072 entries, up to 7 drafts, 27 and 31 us, 16 35 and 41, 32 of 65536 39 and 43, 128 of
// 32000 49 and 60, 64 of 65536 54 and 51.  By parts of up to 4096, 8192, 16384: 64 of 131072 76,
// 74, 79, 128 with up to 3 drafts 96, 92, 115, 256 with up to one 132, 123, 176, 512 of 50257 164,
// 166, 222, 256 of 32000 96, 70, 67.  Past that only where a launch would not hold them.
Cut cut_of(int64_t drafts, int64_t requests, int64_t vocab) {
    const int64_t rows = 2 * drafts + requests;
    int64_t chunk = 65536;
    while (chunk > 2048 && rows * ((vocab + chunk - 1) / chunk) < 4096) chunk /= 2;
    const auto least = [&](int64_t size, int64_t most, int64_t unit) {
        const int64_t n = (vocab + most - 1) / most;
        return size < n ? (n + unit - 1) / unit * unit : size;
    };
    chunk = least(chunk, kMostChunks, 2048);
    int64_t part = kPart;
    while (requests * ((vocab + part - 1) / part) > (part < 8192 ? 512 : kMostBlocks)) part *= 2;
    part = least(part, kMostParts, kPart);
    return {(uint32_t)chunk, (uint32_t)((vocab + chunk - 1) / chunk), (uint32_t)part,
            (uint32_t)((vocab + part - 1) / part)};
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
    s.arrived = s.sums + requests * c.parts * (kOpThreads / 64) * 16;
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
    if ((2 * q.num_drafts + q.num_requests) * cut.chunks > kMostBlocks ||
        q.num_requests * cut.parts > kMostBlocks)
        return SEGTOPK_NOT_SUPPORTED;
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
    a.part = cut.part;
    a.parts = cut.parts;
    const unsigned rows = a.drafts + a.requests + (has_draft ? a.drafts : 0u);
    return with_type(q.target.type, [&](auto v) -> int {
        using T = decltype(v);
        const T *target = static_cast<const T *>(q.target.data);
        const T *draft = has_draft ? static_cast<const T *>(q.draft.data) : nullptr;
        // Four pieces a thread at once; one where a chunk has no more than four, so that nobody
        // adds up nothing (one request of 32003: 14.7 against 12.4 us a call; 30 of 93639, chunks
        // of three pieces a thread, 44 against 36).
        const auto stats = [&](auto kernel) {
            return launch(kernel, dim3(rows * a.chunks), kOpThreads, stream, 0, target, draft, a);
        };
        const bool few = a.chunk <= 4 * kOpThreads * Piece<T>::N;
        if ((few ? stats(stats_kernel<T, 1>) : stats(stats_kernel<T, 4>)) != hipSuccess)
            return SEGTOPK_HIP_ERROR;
        return status(launch(pick_kernel<T>, dim3(a.requests * a.parts), kOpThreads, stream, 0,
                             target, draft, a));
    });
}
