// policy_loss.hip -- the clipped policy loss with a KL term, over the logits of
// sampled tokens, and its gradient.
//
// For a row t with sampled token y, z = logits / temperature:
//   lse  = m + log sum exp(z - m),  m = max z;   lp = z[y] - lse
//   r    = exp(lp - old),  A the advantage
//   term = -min(r A, clamp(r, 1 - low, 1 + high) A)
//          + kl (exp(ref - lp) - (ref - lp) - 1)
//   loss = sum_t weight_t term_t,  weight_t = 1 / (answers * live rows of its answer)
//   d term / d lp = -(r A where the unclipped side is the minimum, else 0)
//                   + kl (1 - exp(ref - lp))
//   dlogits[c] = weight_t (d term / d lp) (1[c = y] - exp(z[c] - lse)) / temperature
// A row without a token in [0, vocab), or in no answer, counts for nothing: its
// gradient is zero.
//
//   weight_kernel  one workgroup an answer: its live rows, and their weights
//   row_kernel     one workgroup a row: maximum and sum in one pass (32 bits),
//                  then, where asked for, the gradient in a second
//   total_kernel   the sum of the rows' terms in 64 bits, in one fixed order
#include "ops_common.h"

namespace segtopk_ops {
namespace {

struct LossArgs {
    int64_t stride, dstride;
    const void *token_ids;
    const float *old_logp, *ref_logp, *advantages;
    float *logp;
    const float *weight;  // [tokens], 0 for a row that counts for nothing
    double *term;         // [tokens]
    uint32_t tokens, vocab, wide;
    float clip_low, clip_high, kl_coef, inv_temperature, grad_scale;
};

__device__ inline int64_t token_of(const void *ids, uint32_t wide, uint32_t t) {
    return wide ? static_cast<const int64_t *>(ids)[t]
                : (int64_t) static_cast<const int32_t *>(ids)[t];
}

__global__ __launch_bounds__(kOpThreads) void weight_kernel(const void *ids, uint32_t wide,
                                                            uint32_t tokens, uint32_t vocab,
                                                            const int64_t *offsets,
                                                            uint32_t segments, float *weight) {
    __shared__ uint32_t live;
    const auto at = [&](uint32_t s) {  // offsets outside the rows are cut
        const int64_t v = offsets[s];
        return (uint32_t)(v < 0 ? 0 : v > (int64_t)tokens ? (int64_t)tokens : v);
    };
    const uint32_t s = blockIdx.x;
    const uint32_t b = at(s), e = at(s + 1);
    if (threadIdx.x == 0) live = 0u;
    __syncthreads();
    uint32_t n = 0;
    for (uint32_t t = b + threadIdx.x; t < e; t += kOpThreads) {
        const int64_t y = token_of(ids, wide, t);
        n += y >= 0 && y < (int64_t)vocab;
    }
    if (n) atomicAdd(&live, n);
    __syncthreads();
    const float w = 1.0f / ((float)segments * (float)live);
    for (uint32_t t = b + threadIdx.x; t < e; t += kOpThreads) {
        const int64_t y = token_of(ids, wide, t);
        weight[t] = y >= 0 && y < (int64_t)vocab ? w : 0.0f;
    }
    if (s == 0)
        for (uint32_t t = threadIdx.x; t < b; t += kOpThreads) weight[t] = 0.0f;
    if (s == segments - 1)
        for (uint32_t t = e + threadIdx.x; t < tokens; t += kOpThreads) weight[t] = 0.0f;
}

constexpr int kRowThreads = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Running maximum m (of the scaled logits, base 2) and sum of 2^(z - m).
struct Stat {
    float m, s;
};
__device__ inline float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ inline Stat join(Stat a, Stat b) {
    const float m = fmaxf(a.m, b.m), o = shift_of(m);
    return {m, a.s * exp2f(a.m - o) + b.s * exp2f(b.m - o)};
}

template <class T, bool GRAD>
__global__ __launch_bounds__(kRowThreads) void row_kernel(const T *logits, T *dlogits,
                                                          LossArgs a) {
    using P = Piece<T>;
    const uint32_t t = blockIdx.x, i = threadIdx.x;
    const float weight = a.weight[t];
    const T *row = logits + (int64_t)t * a.stride;
    T *grad = GRAD ? dlogits + (int64_t)t * a.dstride : nullptr;
    const uint32_t pieces = a.vocab / P::N;
    const float scale = a.inv_temperature * kLog2e;
    float slope = 0.0f, lse = 0.0f;
    uint32_t token = 0;
    if (weight != 0.0f) {
        token = (uint32_t)token_of(a.token_ids, a.wide, t);
        const float zy = (float)row[token] * scale;  // read before the gradient may overwrite it
        Stat st{-INFINITY, 0.0f};
        for (uint32_t u = i; u < pieces; u += kRowThreads) {
            const typename P::f32 z = widen<T>(load_piece(row + (size_t)u * P::N)) * scale;
            float m = st.m;
#pragma unroll
            for (int j = 0; j < P::N; ++j) m = fmaxf(m, z[j]);
            const float o = shift_of(m);
            st.s *= exp2f(st.m - o);
#pragma unroll
            for (int j = 0; j < P::N; ++j) st.s += exp2f(z[j] - o);
            st.m = m;
        }
        for (uint32_t c = pieces * P::N + i; c < a.vocab; c += kRowThreads)
            st = join(st, Stat{(float)row[c] * scale, 1.0f});
#pragma unroll
        for (int d = 32; d; d >>= 1)
            st = join(st, Stat{__shfl_xor(st.m, d), __shfl_xor(st.s, d)});
        __shared__ Stat part[kRowThreads / 64];
        if ((i & 63u) == 0) part[i >> 6] = st;
        __syncthreads();
        st = part[0];
        for (int w = 1; w < kRowThreads / 64; ++w) st = join(st, part[w]);
        if (st.m != -INFINITY) {
            lse = st.m + log2f(st.s);
            const float lp = (zy - lse) * kLn2;
            const float adv = a.advantages[t], ratio = expf(lp - a.old_logp[t]);
            const float clipped = fminf(fmaxf(ratio, 1.0f - a.clip_low), 1.0f + a.clip_high);
            const bool free = ratio * adv <= clipped * adv;
            float term = -(free ? ratio : clipped) * adv;
            slope = free ? -ratio * adv : 0.0f;
            if (a.kl_coef != 0.0f) {
                const float apart = a.ref_logp[t] - lp, e = expf(apart);
                term += a.kl_coef * (e - apart - 1.0f);
                slope += a.kl_coef * (1.0f - e);
            }
            slope *= weight * a.inv_temperature * a.grad_scale;
            if (i == 0) {
                a.logp[t] = lp;
                a.term[t] = (double)term * (double)weight;
            }
        } else if (i == 0) {  // nothing but -inf: no distribution, and no loss
            a.logp[t] = 0.0f;
            a.term[t] = 0.0;
        }
    } else if (i == 0) {
        a.logp[t] = 0.0f;
        a.term[t] = 0.0;
    }
    if (!GRAD) return;
    if (slope == 0.0f) {
        for (uint32_t u = i; u < pieces; u += kRowThreads)
            store_piece(grad + (size_t)u * P::N, (typename P::vec)(T)0.0f);
        for (uint32_t c = pieces * P::N + i; c < a.vocab; c += kRowThreads) grad[c] = (T)0.0f;
        return;
    }
    for (uint32_t u = i; u < pieces; u += kRowThreads) {
        const typename P::f32 z = widen<T>(load_piece(row + (size_t)u * P::N)) * scale;
        typename P::f32 g;
#pragma unroll
        for (int j = 0; j < P::N; ++j) {
            const float p = exp2f(z[j] - lse);
            g[j] = slope * ((u * P::N + j == token ? 1.0f : 0.0f) - p);
        }
        store_piece(grad + (size_t)u * P::N, narrow<T>(g));
    }
    for (uint32_t c = pieces * P::N + i; c < a.vocab; c += kRowThreads)
        grad[c] = (T)(slope * ((c == token ? 1.0f : 0.0f) - exp2f((float)row[c] * scale - lse)));
}

__global__ __launch_bounds__(1024) void total_kernel(const double *term, uint32_t n, float *loss) {
    __shared__ double part[16];
    double v = 0.0;
    for (uint32_t t = threadIdx.x; t < n; t += 1024u) v += term[t];
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) v += part[w];
        *loss = (float)v;
    }
}

__global__ void no_answers_kernel(float *weight, uint32_t n) {
    for (uint32_t t = blockIdx.x * blockDim.x + threadIdx.x; t < n; t += gridDim.x * blockDim.x)
        weight[t] = 0.0f;
}

size_t term_bytes(int64_t tokens) { return ((size_t)tokens * 8 + 255) & ~(size_t)255; }

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
    return (int64_t)(term_bytes(tokens) + (size_t)tokens * 4);
}

extern "C" int segtopk_policy_loss(const segtopk_policy_loss_args *args, void *workspace,
                                   int64_t workspace_bytes, hipStream_t stream) {
    if (!args) return SEGTOPK_INVALID_ARGUMENT;
    const segtopk_policy_loss_args &q = *args;
    if (!good_loss_sizes(q.tokens, q.vocab, q.num_segments)) return SEGTOPK_INVALID_ARGUMENT;
    const bool grad = q.dlogits.data != nullptr;
    const int ib = index_bytes(q.id_type);
    // The comparisons are false for NaN, which is refused with the rest.
    if (!(q.clip_low >= 0.0f && q.clip_low <= 1.0f) || !(q.clip_high >= 0.0f) ||
        !(q.kl_coef >= 0.0f) || !(q.temperature > 0.0f) || !(q.temperature < INFINITY) ||
        !(q.grad_scale - q.grad_scale == 0.0f) || !(q.kl_coef < INFINITY) || !ib)
        return SEGTOPK_INVALID_ARGUMENT;
    if (!q.loss || !aligned(q.loss, 4)) return SEGTOPK_INVALID_ARGUMENT;
    if (q.num_segments && (!q.segment_offsets || !aligned(q.segment_offsets, 8)))
        return SEGTOPK_INVALID_ARGUMENT;
    if (q.tokens) {
        if (!good_rows(&q.logits, q.vocab) || !q.token_ids || !aligned(q.token_ids, ib) ||
            !q.old_logp || !aligned(q.old_logp, 4) || !q.advantages || !aligned(q.advantages, 4) ||
            !q.logp || !aligned(q.logp, 4) || !aligned(q.ref_logp, 4) ||
            (q.kl_coef != 0.0f && !q.ref_logp))
            return SEGTOPK_INVALID_ARGUMENT;
        if (grad && (!good_rows(&q.dlogits, q.vocab) || q.dlogits.type != q.logits.type))
            return SEGTOPK_INVALID_ARGUMENT;
    }
    const size_t need = term_bytes(q.tokens) + (size_t)q.tokens * 4;
    if (need && (!workspace || !aligned(workspace, 256))) return SEGTOPK_INVALID_ARGUMENT;
    if (workspace_bytes < 0 || (size_t)workspace_bytes < need) return SEGTOPK_SCRATCH_TOO_SMALL;

    double *term = static_cast<double *>(workspace);
    float *weight = reinterpret_cast<float *>(static_cast<char *>(workspace) + term_bytes(q.tokens));
    LossArgs a{};
    a.stride = q.logits.stride;
    a.dstride = q.dlogits.stride;
    a.token_ids = q.token_ids;
    a.old_logp = q.old_logp;
    a.ref_logp = q.ref_logp;
    a.advantages = q.advantages;
    a.logp = q.logp;
    a.weight = weight;
    a.term = term;
    a.tokens = (uint32_t)q.tokens;
    a.vocab = (uint32_t)q.vocab;
    a.wide = q.id_type == SEGTOPK_KEY_I64;
    a.clip_low = q.clip_low;
    a.clip_high = q.clip_high;
    a.kl_coef = q.kl_coef;
    a.inv_temperature = 1.0f / q.temperature;
    a.grad_scale = q.grad_scale;
    hipError_t err;
    if (q.tokens) {
        if (q.num_segments)
            hipLaunchKernelGGL(weight_kernel, dim3((unsigned)q.num_segments), dim3(kOpThreads), 0,
                               stream, q.token_ids, a.wide, a.tokens, a.vocab, q.segment_offsets,
                               (uint32_t)q.num_segments, weight);
        else
            hipLaunchKernelGGL(no_answers_kernel, dim3(64), dim3(kOpThreads), 0, stream, weight,
                               a.tokens);
        if ((err = hipGetLastError()) != hipSuccess) return SEGTOPK_HIP_ERROR;
        const int st = with_type(q.logits.type, [&](auto v) {
            using T = decltype(v);
            const T *in = static_cast<const T *>(q.logits.data);
            T *out = static_cast<T *>(q.dlogits.data);
            if (grad)
                hipLaunchKernelGGL((row_kernel<T, true>), dim3(a.tokens), dim3(kRowThreads), 0,
                                   stream, in, out, a);
            else
                hipLaunchKernelGGL((row_kernel<T, false>), dim3(a.tokens), dim3(kRowThreads), 0,
                                   stream, in, out, a);
            return status(hipGetLastError());
        });
        if (st != SEGTOPK_OK) return st;
    }
    hipLaunchKernelGGL(total_kernel, dim3(1), dim3(1024), 0, stream, term, a.tokens, q.loss);
    return status(hipGetLastError());
}
