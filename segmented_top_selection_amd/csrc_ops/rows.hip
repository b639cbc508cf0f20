// rows.hip -- rows moved between token order and expert order, and rows looked
// up in a table.
//
//   dispatch   rows[position[t, j]] = x[t]
//   combine    out[t] = sum_j w[t, j] rows[position[t, j]]
//   their gradients: dispatch's is combine without weights; combine's sends
//   w[t, j] dout[t] to row position[t, j] and gives
//   dw[t, j] = <dout[t], rows[position[t, j]]>
//   embedding  out[i] = scale * table[id_i]
//
// A slot whose position is not below *kept is dropped: its packed row is
// zero and it adds nothing.  Positions outside [0, tokens * k) are skipped.
//
// All are bound by memory: every row is read once and written once, because
// the work is laid out by token.  A group of `lanes` threads takes one token;
// a thread holds one 16-byte piece of it, so a token's row is read once for
// its k copies (dispatch) or k gradients (combine backward), and a sum over k
// rows stays in registers (32 bits).  Pieces past the last whole one are
// single elements, one to a thread.  What is read once, and outputs of 128 MiB or
// more, go past the caches: left there they are written back while the next
// kernel reads (sort, dispatch and combine of 8192 tokens x 8 x 4096 bf16, the same
// inputs again and again, 263 us, so 216; a kernel that reads the rows right after
// loses 2%).  On new inputs each time the three take 236.
//
// 8192 tokens x 8 x 4096 bf16: dispatch 102 us (5.9 TB/s of what it reads and
// writes), combine 104 (5.8), its gradient 219 (5.2); a 4 GiB copy reaches 4.7.
// Lookup of 32768 rows of 4096 bf16, new rows each time: 70 us (5.1 TB/s).
#include <type_traits>

#include "ops_common.h"

namespace segtopk_ops {
namespace {

// How a row of `width` elements is cut up: `pieces` whole pieces, then
// single elements, together `units`; a group of `lanes` (a power of two)
// threads walks them.
struct Cut {
    uint32_t pieces, units, lanes;
};

constexpr int kSlotsAtOnce = 8;  // a token's slots that a thread works on together, at most

// For k up to four, kernels of four: 8192 tokens x 2 x 4096 bf16, both gradients,
// 96 -> 88 us, 1500 x 2 x 512 9.4 -> 7.7.
constexpr int kFewSlots = 4;

struct Slots {
    const int32_t *position;  // [tokens][k]
    const int64_t *kept;      // or nullptr: all
    uint32_t tokens, k, count;  // count = tokens * k
};

__device__ inline uint32_t kept_of(const Slots &s) {
    if (!s.kept) return s.count;
    const int64_t v = *s.kept;
    return v < 0 ? 0u : v < (int64_t)s.count ? (uint32_t)v : s.count;
}

// A value that all lanes of a wave share, in a scalar register.  Rows of 64
// units or more have a wave to themselves (ONE): what belongs to the token is
// the wave's then, which takes its addresses out of the vector registers.
template <bool ONE> __device__ inline uint32_t shared(uint32_t v) {
    return ONE ? (uint32_t)__builtin_amdgcn_readfirstlane((int)v) : v;
}
template <bool ONE> __device__ inline float shared(float v) {
    return ONE ? __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))) : v;
}

template <class T, bool ONE, bool STREAM>
__global__ __launch_bounds__(kOpThreads) void dispatch_kernel(const T *__restrict__ x, int64_t xs,
                                                              T *__restrict__ rows, int64_t rs,
                                                              Slots s, Cut c) {
    using P = Piece<T>;
    const uint32_t kept = kept_of(s), per = kOpThreads / c.lanes;
    for (uint32_t token = blockIdx.x * per + shared<ONE>(threadIdx.x / c.lanes); token < s.tokens;
         token += gridDim.x * per) {
        const int32_t *pos = s.position + (size_t)token * s.k;
        const T *src = x + (int64_t)token * xs;
        for (uint32_t u = blockIdx.y * c.lanes + (threadIdx.x & (c.lanes - 1u)); u < c.units;
             u += gridDim.y * c.lanes) {
            const bool whole = u < c.pieces;
            const size_t at = whole ? (size_t)u * P::N : (size_t)c.pieces * P::N + (u - c.pieces);
            typename P::vec v = (typename P::vec)(T)0.0f;
            if (whole) v = load_piece(src + at);
            else v[0] = src[at];
            for (uint32_t j0 = 0; j0 < s.k; j0 += kSlotsAtOnce) {
                uint32_t p[kSlotsAtOnce];
#pragma unroll
                for (int j = 0; j < kSlotsAtOnce; ++j)
                    p[j] = shared<ONE>(j0 + j < s.k ? (uint32_t)pos[j0 + j] : 0xFFFFFFFFu);
#pragma unroll
                for (int j = 0; j < kSlotsAtOnce; ++j) {
                    if (p[j] >= s.count) continue;
                    T *dst = rows + (int64_t)p[j] * rs + at;
                    const typename P::vec o = p[j] < kept ? v : (typename P::vec)(T)0.0f;
                    if (whole) store_piece<STREAM>(dst, o);
                    else *dst = o[0];
                }
            }
        }
    }
}

template <class T, class W, bool ONE, int SLOTS>
__global__ __launch_bounds__(kOpThreads) void combine_kernel(const T *__restrict__ rows,
                                                             int64_t rs, T *__restrict__ out,
                                                             int64_t os,
                                                             const W *__restrict__ weights,
                                                             Slots s, Cut c) {
    using P = Piece<T>;
    const uint32_t kept = kept_of(s), per = kOpThreads / c.lanes;
    for (uint32_t token = blockIdx.x * per + shared<ONE>(threadIdx.x / c.lanes); token < s.tokens;
         token += gridDim.x * per) {
        const int32_t *pos = s.position + (size_t)token * s.k;
        const W *wt = weights ? weights + (size_t)token * s.k : nullptr;
        T *dst = out + (int64_t)token * os;
        for (uint32_t u = blockIdx.y * c.lanes + (threadIdx.x & (c.lanes - 1u)); u < c.units;
             u += gridDim.y * c.lanes) {
            if (u < c.pieces) {
                typename P::f32 acc = 0.0f;
                // The rows of up to SLOTS slots are in flight together.
                for (uint32_t j0 = 0; j0 < s.k; j0 += SLOTS) {
                    uint32_t p[SLOTS];
                    float w[SLOTS];
                    typename P::vec v[SLOTS];
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j) {
                        const bool here = j0 + j < s.k;
                        p[j] = shared<ONE>(here ? (uint32_t)pos[j0 + j] : 0xFFFFFFFFu);
                        w[j] = shared<ONE>(here && wt ? (float)wt[j0 + j] : 1.0f);
                    }
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j) {
                        v[j] = (typename P::vec)(T)0.0f;
                        if (p[j] < kept)
                            v[j] = load_piece<true>(rows + (int64_t)p[j] * rs + (size_t)u * P::N);
                    }
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j)
                        if (p[j] < kept) acc += w[j] * widen<T>(v[j]);
                }
                store_piece(dst + (size_t)u * P::N, narrow<T>(acc));
            } else {
                const size_t at = (size_t)c.pieces * P::N + (u - c.pieces);
                float acc = 0.0f;
                for (uint32_t j = 0; j < s.k; ++j) {
                    const uint32_t p = shared<ONE>((uint32_t)pos[j]);
                    if (p >= kept) continue;
                    acc += (wt ? (float)wt[j] : 1.0f) * (float)rows[(int64_t)p * rs + at];
                }
                dst[at] = (T)acc;
            }
        }
    }
}

template <class T, class W, bool STREAM, int SLOTS>
__global__ __launch_bounds__(kOpThreads) void combine_backward_kernel(
    const T *__restrict__ dout, int64_t ds, const T *__restrict__ rows, int64_t rs,
    T *__restrict__ drows, int64_t drs, const W *__restrict__ weights, W *__restrict__ dweights,
    Slots s, Cut c) {
    using P = Piece<T>;
    __shared__ float part[kOpThreads / 64][SLOTS];
    const uint32_t lane = threadIdx.x & (c.lanes - 1u);  // lanes: 64 or all threads
    const uint32_t kept = kept_of(s), per = kOpThreads / c.lanes;
    for (uint32_t first = blockIdx.x * per; first < s.tokens; first += gridDim.x * per) {
        const uint32_t token = first + shared<true>(threadIdx.x / c.lanes);
        const bool live = token < s.tokens;
        const T *g = dout + (int64_t)token * ds;
        for (uint32_t j0 = 0; j0 < s.k; j0 += SLOTS) {
            const uint32_t m = min((uint32_t)SLOTS, s.k - j0);
            uint32_t p[SLOTS];
            float w[SLOTS], dot[SLOTS];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const bool here = live && (uint32_t)j < m;
                const size_t i = (size_t)token * s.k + j0 + j;
                p[j] = shared<true>(here ? (uint32_t)s.position[i] : 0xFFFFFFFFu);
                w[j] = shared<true>(here && weights ? (float)weights[i] : 1.0f);
                if (p[j] >= kept) w[j] = 0.0f;
                dot[j] = 0.0f;
            }
            if (live)
                for (uint32_t u = lane; u < c.units; u += c.lanes) {
                    if (u < c.pieces) {
                        const size_t at = (size_t)u * P::N;
                        const typename P::f32 d = widen<T>(load_piece(g + at));
                        typename P::vec y[SLOTS];
#pragma unroll
                        for (int j = 0; j < SLOTS; ++j) {
                            y[j] = (typename P::vec)(T)0.0f;
                            if (p[j] < kept && dweights)
                                y[j] = load_piece<true>(rows + (int64_t)p[j] * rs + at);
                        }
#pragma unroll
                        for (int j = 0; j < SLOTS; ++j) {
                            if (p[j] >= s.count) continue;
                            typename P::f32 r = 0.0f;
                            if (p[j] < kept) r = w[j] * d;
                            store_piece<STREAM>(drows + (int64_t)p[j] * drs + at, narrow<T>(r));
                        }
#pragma unroll
                        for (int j = 0; j < SLOTS; ++j) {
                            if (p[j] >= kept) continue;
                            const typename P::f32 v = widen<T>(y[j]);
#pragma unroll
                            for (int i = 0; i < P::N; ++i) dot[j] += d[i] * v[i];
                        }
                    } else {
                        const size_t at = (size_t)c.pieces * P::N + (u - c.pieces);
                        const float d = (float)g[at];
#pragma unroll
                        for (int j = 0; j < SLOTS; ++j) {
                            if (p[j] >= s.count) continue;
                            if (p[j] < kept && dweights)
                                dot[j] += d * (float)rows[(int64_t)p[j] * rs + at];
                            drows[(int64_t)p[j] * drs + at] = p[j] < kept ? (T)(w[j] * d) : (T)0.0f;
                        }
                    }
                }
            if (!dweights) continue;
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) dot[j] = wave_sum(dot[j]);
            if (c.lanes == 64u) {
                if (live && lane == 0)
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j)
                        if ((uint32_t)j < m) dweights[(size_t)token * s.k + j0 + j] = (W)dot[j];
            } else {
                if ((threadIdx.x & 63u) == 0)
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j) part[threadIdx.x >> 6][j] = dot[j];
                __syncthreads();
                if (threadIdx.x < m) {
                    float v = 0.0f;
                    for (int i = 0; i < kOpThreads / 64; ++i) v += part[i][threadIdx.x];
                    dweights[(size_t)token * s.k + j0 + threadIdx.x] = (W)v;
                }
                __syncthreads();
            }
        }
    }
}

// A group of threads takes ROWS rows, so that a thread has that many loads in
// flight.
template <class T, class I, int ROWS, bool STREAM, int THREADS>
__global__ __launch_bounds__(THREADS) void embedding_kernel(const T *__restrict__ table,
                                                               int64_t ts, T *__restrict__ out,
                                                               int64_t os,
                                                               const I *__restrict__ ids,
                                                               uint32_t n, int64_t num_rows,
                                                               float scale, Cut c) {
    using P = Piece<T>;
    const uint32_t per = (uint32_t)THREADS / c.lanes;
    for (uint32_t i0 = blockIdx.x * per * ROWS + threadIdx.x / c.lanes; i0 < n;
         i0 += gridDim.x * per * ROWS) {
        int64_t id[ROWS];  // -1: a row of zeros
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const uint32_t i = i0 + r * per;
            id[r] = i < n ? (int64_t)ids[i] : -1;
            if (id[r] >= num_rows) id[r] = -1;
        }
        for (uint32_t u = blockIdx.y * c.lanes + (threadIdx.x & (c.lanes - 1u)); u < c.units;
             u += gridDim.y * c.lanes) {
            if (u < c.pieces) {
                const size_t at = (size_t)u * P::N;
                typename P::vec v[ROWS];
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    v[r] = (typename P::vec)(T)0.0f;
                    if (id[r] >= 0) v[r] = load_piece(table + id[r] * ts + at);
                }
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    if (i0 + r * per < n)
                        store_piece<STREAM>(
                            out + (int64_t)(i0 + r * per) * os + at,
                            id[r] >= 0 ? narrow<T>(scale * widen<T>(v[r])) : v[r]);
            } else {
                const size_t at = (size_t)c.pieces * P::N + (u - c.pieces);
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    if (i0 + r * per < n)
                        out[(int64_t)(i0 + r * per) * os + at] =
                            id[r] >= 0 ? (T)(scale * (float)table[id[r] * ts + at]) : (T)0.0f;
            }
        }
    }
}

constexpr int64_t kManyPieces = 4 * 256 * 2048;  // four for each thread that 256 CUs hold

Cut cut_of(int64_t width, int elem_bytes, uint32_t threads = kOpThreads) {
    const int64_t n = 16 / elem_bytes;
    Cut c;
    c.pieces = (uint32_t)(width / n);
    c.units = (uint32_t)(width / n + width % n);
    c.lanes = 8;
    while (c.lanes < threads && c.lanes < c.units) c.lanes <<= 1;
    return c;
}

// A launch holds fewer than 2^32 threads in a direction; the kernels loop over
// the tokens that are left.
unsigned blocks_of(int64_t tokens, const Cut &c, uint32_t threads = kOpThreads) {
    const int64_t per = threads / c.lanes, most = ((int64_t)1 << 30) / threads;
    const int64_t n = (tokens + per - 1) / per;
    return (unsigned)(n < most ? n : most);
}

dim3 grid_of(int64_t tokens, const Cut &c, uint32_t threads = kOpThreads) {
    const uint32_t y = (c.units + c.lanes - 1) / c.lanes;
    return dim3(blocks_of(tokens, c, threads), y < 65535u ? y : 65535u);
}

bool good_slots(int64_t tokens, int64_t k, int64_t width, const int32_t *position,
                const int64_t *kept) {
    return tokens >= 0 && k >= 1 && width >= 1 && width <= INT32_MAX && k <= INT32_MAX &&
           tokens <= INT32_MAX / k && (tokens == 0 || position) && aligned(position, 4) &&
           aligned(kept, 8);
}

Slots slots_of(int64_t tokens, int64_t k, const int32_t *position, const int64_t *kept) {
    return Slots{position, kept, (uint32_t)tokens, (uint32_t)k, (uint32_t)(tokens * k)};
}

// Weights are absent, of 32 bits, or of the rows' type.
bool good_weights(const void *weights, int32_t weight_type, int row_type) {
    if (!weights) return true;
    return (weight_type == SEGTOPK_KEY_F32 || weight_type == row_type) &&
           aligned(weights, element_bytes(weight_type));
}

}  // namespace
}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int segtopk_dispatch_rows(const segtopk_rows *x, const segtopk_rows *rows,
                                     int64_t tokens, int64_t k, int64_t width,
                                     const int32_t *position, const int64_t *kept,
                                     hipStream_t stream) {
    if (!good_slots(tokens, k, width, position, kept)) return SEGTOPK_INVALID_ARGUMENT;
    if (tokens == 0) return SEGTOPK_OK;
    if (!good_rows(x, width) || !good_rows(rows, width) || x->type != rows->type)
        return SEGTOPK_INVALID_ARGUMENT;
    return with_type(x->type, [&](auto t) {
        using T = decltype(t);
        const Cut c = cut_of(width, sizeof(T));
        const auto go = [&](auto kernel) {
            return status(launch(kernel, grid_of(tokens, c), kOpThreads, stream, 0,
                                 static_cast<const T *>(x->data), x->stride,
                                 static_cast<T *>(rows->data), rows->stride,
                                 slots_of(tokens, k, position, kept), c));
        };
        if (c.lanes < 64u) return go(dispatch_kernel<T, false, false>);
        return streams(tokens * k * width * (int64_t)sizeof(T)) ? go(dispatch_kernel<T, true, true>)
                                                                : go(dispatch_kernel<T, true, false>);
    });
}

extern "C" int segtopk_combine_rows(const segtopk_rows *rows, const segtopk_rows *out,
                                    const void *weights, int32_t weight_type, int64_t tokens,
                                    int64_t k, int64_t width, const int32_t *position,
                                    const int64_t *kept, hipStream_t stream) {
    if (!good_slots(tokens, k, width, position, kept)) return SEGTOPK_INVALID_ARGUMENT;
    if (tokens == 0) return SEGTOPK_OK;
    if (!good_rows(rows, width) || !good_rows(out, width) || rows->type != out->type ||
        !good_weights(weights, weight_type, rows->type))
        return SEGTOPK_INVALID_ARGUMENT;
    return with_type(rows->type, [&](auto t) {
        using T = decltype(t);
        const Cut c = cut_of(width, sizeof(T));
        const auto with = [&](auto kernel, auto w) {
            return status(launch(kernel, grid_of(tokens, c), kOpThreads, stream, 0,
                                 static_cast<const T *>(rows->data), rows->stride,
                                 static_cast<T *>(out->data), out->stride,
                                 static_cast<const decltype(w) *>(weights),
                                 slots_of(tokens, k, position, kept), c));
        };
        const auto go = [&](auto w) {
            using W = decltype(w);
            const bool one = c.lanes >= 64u;
            if (k <= kFewSlots)
                return one ? with(combine_kernel<T, W, true, kFewSlots>, w)
                           : with(combine_kernel<T, W, false, kFewSlots>, w);
            return one ? with(combine_kernel<T, W, true, kSlotsAtOnce>, w)
                       : with(combine_kernel<T, W, false, kSlotsAtOnce>, w);
        };
        return weights && weight_type != SEGTOPK_KEY_F32 ? go(t) : go(float{});
    });
}

extern "C" int segtopk_combine_rows_backward(const segtopk_rows *dout, const segtopk_rows *rows,
                                             const segtopk_rows *drows, const void *weights,
                                             void *dweights, int32_t weight_type, int64_t tokens,
                                             int64_t k, int64_t width, const int32_t *position,
                                             const int64_t *kept, hipStream_t stream) {
    if (!good_slots(tokens, k, width, position, kept)) return SEGTOPK_INVALID_ARGUMENT;
    if (tokens == 0) return SEGTOPK_OK;
    if (!good_rows(dout, width) || !good_rows(drows, width) || dout->type != drows->type ||
        !good_weights(weights, weight_type, dout->type) ||
        !good_weights(dweights, weight_type, dout->type))
        return SEGTOPK_INVALID_ARGUMENT;
    // Without the weights' gradient the rows are not read.
    if (dweights && (!good_rows(rows, width) || rows->type != dout->type))
        return SEGTOPK_INVALID_ARGUMENT;
    return with_type(dout->type, [&](auto t) {
        using T = decltype(t);
        Cut c = cut_of(width, sizeof(T));
        // A row of more than 128 units by a wave or by a workgroup, us of this kernel, bf16
        // (k = 2, 4, 8 in turn).  Few tokens leave waves idle: 256 x 1410 6.0, 7.5, 13.0
        // and 4.5, 5.7, 8.8; 1024 x 2048 8.5, 12.7, 19.6 and 6.7, 10.2, 17.1.  From 2048
        // on the waves fill the device: 2048 x 1410 10.1, 15.9, 27.0 and 12.4, 18.6, 31.7;
        // 4096 x 1410 14.4, 23.6, 47.4 and 19.5, 30.2, 61.3.  At the widest, 256 units, it
        // depends on k: 4096 x 2048 16.7, 28.7, 69.1 and 18.1, 28.8, 57.4.  Wider rows
        // are a workgroup's: 4096 x 4096 31.4 and 31.2 (k = 2), 123 and 112 (k = 8).  Up to
        // 128 units a wave holds the row in two rounds: 2048 x 1000 7.1 and 9.3 (k = 2).
        const bool wide = c.units > 256u || (c.units > 128u && tokens < 2048);
        c.lanes = wide ? (uint32_t)kOpThreads : 64u;
        const bool past = streams(tokens * k * width * (int64_t)sizeof(T));
        const auto with = [&](auto kernel, auto w) {
            using W = decltype(w);
            return status(launch(kernel, dim3(blocks_of(tokens, c)), kOpThreads, stream, 0,
                                 static_cast<const T *>(dout->data), dout->stride,
                                 static_cast<const T *>(rows ? rows->data : nullptr),
                                 rows ? rows->stride : 0, static_cast<T *>(drows->data),
                                 drows->stride, static_cast<const W *>(weights),
                                 static_cast<W *>(dweights), slots_of(tokens, k, position, kept), c));
        };
        const auto go = [&](auto w) {
            using W = decltype(w);
            if (k <= kFewSlots)
                return past ? with(combine_backward_kernel<T, W, true, kFewSlots>, w)
                            : with(combine_backward_kernel<T, W, false, kFewSlots>, w);
            return past ? with(combine_backward_kernel<T, W, true, kSlotsAtOnce>, w)
                        : with(combine_backward_kernel<T, W, false, kSlotsAtOnce>, w);
        };
        return (weights || dweights) && weight_type != SEGTOPK_KEY_F32 ? go(t) : go(float{});
    });
}

extern "C" int segtopk_embedding_rows(const segtopk_rows *table, const segtopk_rows *out,
                                      const void *ids, int32_t id_type, int64_t n,
                                      int64_t num_rows, int64_t width, float scale,
                                      hipStream_t stream) {
    const int ib = index_bytes(id_type);
    if (!ib || n < 0 || n > INT32_MAX || num_rows < 0 || num_rows >= INT32_MAX || width < 1 ||
        width > INT32_MAX)
        return SEGTOPK_INVALID_ARGUMENT;
    if (n == 0) return SEGTOPK_OK;
    if (!ids || !aligned(ids, ib) || !good_rows(out, width)) return SEGTOPK_INVALID_ARGUMENT;
    if (num_rows && (!good_rows(table, width) || table->type != out->type))
        return SEGTOPK_INVALID_ARGUMENT;
    return with_type(out->type, [&](auto t) {
        using T = decltype(t);
        const int64_t units = cut_of(width, sizeof(T)).units;
        const auto go = [&](auto i, auto rows, auto past, auto threads) {
            constexpr int kRows = decltype(rows)::value, kThreads = decltype(threads)::value;
            const Cut c = cut_of(width, sizeof(T), kThreads);
            return status(launch(
                embedding_kernel<T, decltype(i), kRows, decltype(past)::value, kThreads>,
                grid_of((n + kRows - 1) / kRows, c, kThreads), kThreads, stream, 0,
                static_cast<const T *>(num_rows ? table->data : nullptr),
                num_rows ? table->stride : 0, static_cast<T *>(out->data), out->stride,
                static_cast<const decltype(i) *>(ids), (uint32_t)n, num_rows, scale, c));
        };
        const auto by_size = [&](auto i) {
            using One = std::integral_constant<int, 1>;
            using Four = std::integral_constant<int, 4>;
            using Small = std::integral_constant<int, kOpThreads>;
            using Large = std::integral_constant<int, 1024>;
            // Four rows a thread once there is work for every wave the device holds.
            if (n * units < kManyPieces) return go(i, One{}, std::false_type{}, Small{});
            // Whole wide rows by one workgroup: 32768 x 4096 bf16 72 us, by two 77.
            const bool wide = units > kOpThreads;
            if (!streams(n * width * (int64_t)sizeof(T)))
                return wide ? go(i, Four{}, std::false_type{}, Large{})
                            : go(i, Four{}, std::false_type{}, Small{});
            return wide ? go(i, Four{}, std::true_type{}, Large{})
                        : go(i, Four{}, std::true_type{}, Small{});
        };
        return id_type == SEGTOPK_KEY_I64 ? by_size(int64_t{}) : by_size(int32_t{});
    });
}
