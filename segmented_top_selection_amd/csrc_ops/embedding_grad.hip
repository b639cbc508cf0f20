// embedding_grad.hip -- the gradient of an embedding table:
//   dtable[v] = scale * sum_{i : id_i = v} dout[i]      (v != padding)
//
// Few tokens take one launch (few_kernel).  Of more, the table is cleared beside
// the sort of the tokens by id (sort_ids.hip), which leaves most of the device
// idle.  Equal ids then lie in runs, and the sorted tokens are cut into chunks of 8
// to 64 rows, so that a frequent token costs no workgroup more than any other:
//   sum_kernel     a workgroup adds up one chunk, 16 bytes of a row to a thread,
//                  in 32 bits; a run inside the chunk goes to its row of the
//                  table at once, a run that crosses the chunk's border leaves a
//                  32-bit partial row
//   finish_kernel  adds the partial rows of a run, chunk by chunk
// Every sum has one fixed order: results are the same every time.
//
// Bound by writing the table, most of whose rows are zeros, and reading dout, or by
// latency where there is little of both (20 tokens, 5000 x 500: 3.9 us):
// 32768 tokens, 131072 x 4096 bf16 take 269 us (1.34 GB, 5.0 TB/s): sort and
// clearing 188, sums 70, finish 8.  Looking up which rows to clear, in sum_kernel,
// took as long.  Of 5003 tokens, 4099 x 1001 f32, the launches' latency is most:
// 8.2 + 7.6 + 5.2 us.
#include "ops_common.h"

namespace segtopk_ops {
namespace {

constexpr uint32_t kMaxChunk = 64;  // rows of dout that a workgroup adds up
constexpr int kRowsAtOnce = 8;      // of which so many are in flight together

struct GradArgs {
    const int32_t *order;
    const uint32_t *sorted;  // ids in order, num_rows for one outside the table
    float *part;             // [chunks][2][width]: the run a chunk ends with, begins with
    uint32_t n, chunk, chunks, num_rows, padding;  // padding >= num_rows: none
    uint32_t pieces, units, cols;  // cols: workgroups side by side over a row
    float scale;
    uint32_t accumulate;
    int64_t width, ds, ts;
};

// Whether the run at sorted place i goes into the table.
__device__ inline bool counts(const GradArgs &a, uint32_t id) {
    return id < a.num_rows && id != a.padding;
}

template <class O> __device__ inline void put(O *dst, float v, const GradArgs &a) {
    v *= a.scale;
    *dst = (O)(a.accumulate ? (float)*dst + v : v);
}

template <class T, class O>
__device__ inline void put_piece(O *dst, typename Piece<T>::f32 v, const GradArgs &a) {
    typedef O vec __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(O))));
    vec *const d = reinterpret_cast<vec *>(dst);
    v *= a.scale;
    if (a.accumulate) v += __builtin_convertvector(*d, typename Piece<T>::f32);
    *d = __builtin_convertvector(v, vec);
}

// Clears rows that are not one piece of memory.
template <class O>
__global__ __launch_bounds__(kOpThreads) void clear_kernel(O *table, uint32_t num_rows,
                                                           int64_t width, int64_t ts) {
    using Q = Piece<O>;
    const int64_t pieces = width / Q::N;
    for (uint32_t v = blockIdx.x; v < num_rows; v += gridDim.x) {
        O *dst = table + (int64_t)v * ts;
        for (int64_t u = threadIdx.x; u < pieces; u += kOpThreads)
            store_piece(dst + u * Q::N, (typename Q::vec)(O)0.0f);
        for (int64_t i = pieces * Q::N + threadIdx.x; i < width; i += kOpThreads) dst[i] = (O)0.0f;
    }
}

template <class T, class O>
__global__ __launch_bounds__(kOpThreads) void sum_kernel(const T *__restrict__ dout, O *table,
                                                         GradArgs a) {
    using P = Piece<T>;
    const uint32_t t = threadIdx.x;
    __shared__ uint32_t id[kMaxChunk], row[kMaxChunk];
    const uint32_t chunk = blockIdx.x / a.cols, col = blockIdx.x % a.cols;
    const uint32_t b = chunk * a.chunk, m = min(a.chunk, a.n - b);
    if (t < m) {
        id[t] = a.sorted[b + t];
        row[t] = (uint32_t)a.order[b + t];
    }
    __syncthreads();
    const bool joins = b && a.sorted[b - 1] == id[0];
    const bool goes_on = b + m < a.n && a.sorted[b + m] == id[m - 1];
    for (uint32_t u = col * kOpThreads + t; u < a.units; u += a.cols * kOpThreads) {
        const bool whole = u < a.pieces;
        const size_t at = whole ? (size_t)u * P::N : (size_t)a.pieces * P::N + (u - a.pieces);
        typename P::f32 acc = 0.0f;
        uint32_t first = 0;  // of the run that is being added
        for (uint32_t i0 = 0; i0 < m; i0 += kRowsAtOnce) {
            uint32_t key[kRowsAtOnce + 1];
            typename P::vec v[kRowsAtOnce];
#pragma unroll
            for (int r = 0; r <= kRowsAtOnce; ++r)  // past the chunk: no id
                key[r] = __builtin_amdgcn_readfirstlane(i0 + r < m ? id[i0 + r] : 0xFFFFFFFFu);
#pragma unroll
            for (int r = 0; r < kRowsAtOnce; ++r) {
                v[r] = (typename P::vec)(T)0.0f;
                if (!counts(a, key[r])) continue;
                const T *src = dout + (int64_t)row[i0 + r] * a.ds + at;
                if (whole) v[r] = load_piece<true>(src);
                else v[r][0] = *src;
            }
#pragma unroll
            for (int r = 0; r < kRowsAtOnce; ++r) {
                if (key[r] == 0xFFFFFFFFu) continue;
                acc += widen<T>(v[r]);
                if (key[r + 1] == key[r]) continue;
                const uint32_t i = i0 + r;
                if (counts(a, key[r])) {
                    const bool head = first == 0 && joins, tail = i + 1 == m && goes_on;
                    if (head || tail) {
                        float *dst = a.part + ((size_t)chunk * 2 + (head ? 1 : 0)) * a.width + at;
                        typedef float mem
                            __attribute__((ext_vector_type(16 / sizeof(T)), aligned(4)));
                        if (whole) *reinterpret_cast<mem *>(dst) = acc;
                        else *dst = acc[0];
                    } else {
                        O *dst = table + (int64_t)key[r] * a.ts + at;
                        if (whole) put_piece<T>(dst, acc, a);
                        else put(dst, acc[0], a);
                    }
                }
                acc = 0.0f;
                first = i + 1;
            }
        }
    }
}

// A workgroup for a chunk that a run starts in and leaves adds the partial rows
// of that run: 64 lanes side by side over the columns, four to a lane, and
// four waves over the chunks, each with eight partial rows in flight.
template <class O>
__global__ __launch_bounds__(kOpThreads) void finish_kernel(O *table, GradArgs a) {
    typedef float f4 __attribute__((ext_vector_type(4)));
    typedef float f4mem __attribute__((ext_vector_type(4), aligned(4)));
    constexpr uint32_t kWaves = kOpThreads / 64;
    const uint32_t chunk = blockIdx.x, b = chunk * a.chunk;
    const uint32_t e = b + a.chunk;  // the next chunk is there: the grid leaves the last one out
    const uint32_t id = a.sorted[e - 1], before = b ? a.sorted[b - 1] : 0xFFFFFFFFu;
    if (!counts(a, id) || a.sorted[e] != id) return;
    if (before == id) return;  // the run started before this chunk
    const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
    // The run reaches into the chunks whose first row is of the same id.
    uint32_t last = chunk + 1;
    while (true) {
        const uint32_t c = last + 1 + lane;
        const uint64_t same = __ballot(c < a.chunks && a.sorted[c * a.chunk] == id);
        const uint32_t run = same == ~0ull ? 64u : (uint32_t)__builtin_ctzll(~same);
        last += run;
        if (run < 64u) break;
    }
    __shared__ f4 part[kWaves][64];
    for (int64_t c0 = (int64_t)blockIdx.y * 256; c0 < a.width; c0 += (int64_t)gridDim.y * 256) {
        const int64_t c = c0 + lane * 4;
        const bool whole = c + 4 <= a.width;
        const uint32_t rest = c < a.width && !whole ? (uint32_t)(a.width - c) : 0u;
        f4 acc = 0.0f;
        for (uint32_t i0 = chunk + w; i0 <= last; i0 += kWaves * kRowsAtOnce) {
            f4 v[kRowsAtOnce];
#pragma unroll
            for (int r = 0; r < kRowsAtOnce; ++r) {
                const uint32_t i = i0 + r * kWaves;
                v[r] = 0.0f;
                if (i > last) continue;
                const float *src = a.part + ((size_t)i * 2 + (i == chunk ? 0 : 1)) * a.width + c;
                if (whole) v[r] = *reinterpret_cast<const f4mem *>(src);
                else if (rest) {
                    v[r][0] = src[0];
                    if (rest > 1) v[r][1] = src[1];
                    if (rest > 2) v[r][2] = src[2];
                }
            }
#pragma unroll
            for (int r = 0; r < kRowsAtOnce; ++r) acc += v[r];
        }
        part[w][lane] = acc;
        __syncthreads();
        if (w == 0) {
            for (uint32_t i = 1; i < kWaves; ++i) acc += part[i][lane];
            O *dst = table + (int64_t)id * a.ts + c;
            if (whole || rest) put(dst, acc[0], a);
            if (whole || rest > 1) put(dst + 1, acc[1], a);
            if (whole || rest > 2) put(dst + 2, acc[2], a);
            if (whole) put(dst + 3, acc[3], a);
        }
        __syncthreads();
    }
}

// Few tokens, in one launch: a workgroup for each token and 64 units of its row
// reads all ids and, if the token is the first of its id, lists the others in
// order and adds up their rows, a quarter to a wave.  The workgroups past those
// clear the rows that no token has, kFewRows or 16 KiB at a time.
constexpr uint32_t kFewTokens = 1024;
constexpr uint32_t kFewRows = 256;

struct FewArgs {
    const void *ids;
    uint32_t wide, cols, sums, rows;  // sums: workgroups that add; rows: that one clears
};

__device__ inline uint32_t few_key(const FewArgs &f, const GradArgs &a, uint32_t i) {
    const int64_t id = f.wide ? static_cast<const int64_t *>(f.ids)[i]
                              : (int64_t) static_cast<const int32_t *>(f.ids)[i];
    return id >= 0 && id < (int64_t)a.num_rows ? (uint32_t)id : a.num_rows;
}

template <class O>
__device__ inline void clear_untouched(O *table, const GradArgs &a, const FewArgs &f,
                                       uint32_t *taken) {
    using Q = Piece<O>;
    const uint32_t t = threadIdx.x;
    const uint32_t pieces = (uint32_t)(a.width / Q::N), rest = (uint32_t)(a.width % Q::N);
    for (uint64_t block = blockIdx.x - f.sums; block * f.rows < a.num_rows;
         block += gridDim.x - f.sums) {
        const uint32_t v0 = (uint32_t)block * f.rows, rows = min(f.rows, a.num_rows - v0);
        taken[t] = 0u;
        __syncthreads();
        for (uint32_t i = t; i < a.n; i += kOpThreads) {
            const uint32_t v = few_key(f, a, i);
            if (v - v0 < rows && v != a.padding) taken[v - v0] = 1u;
        }
        __syncthreads();
        const uint32_t all = rows * pieces;
        for (uint32_t u = t; u < all; u += kOpThreads) {
            const uint32_t r = u / pieces;
            if (!taken[r])
                store_piece(table + (int64_t)(v0 + r) * a.ts + (size_t)(u - r * pieces) * Q::N,
                            (typename Q::vec)(O)0.0f);
        }
        for (uint32_t u = t; u < rows * rest; u += kOpThreads) {
            const uint32_t r = u / rest;
            if (!taken[r])
                table[(int64_t)(v0 + r) * a.ts + (size_t)pieces * Q::N + u % rest] = (O)0.0f;
        }
        __syncthreads();
    }
}

template <class T, class O>
__global__ __launch_bounds__(kOpThreads) void few_kernel(const T *__restrict__ dout, O *table,
                                                         GradArgs a, FewArgs f) {
    using P = Piece<T>;
    constexpr uint32_t kWaves = kOpThreads / 64;
    __shared__ uint32_t key[kFewTokens], list[kFewTokens];
    __shared__ uint32_t found[kWaves], earlier[kWaves];
    __shared__ typename P::f32 part[kWaves][64];
    if (blockIdx.x >= f.sums) return clear_untouched(table, a, f, key);
    const uint32_t t = threadIdx.x, lane = t & 63u, w = t >> 6;
    const uint32_t token = blockIdx.x / f.cols, u = blockIdx.x % f.cols * 64u + lane;
#pragma unroll 4
    for (uint32_t i = t; i < a.n; i += kOpThreads) key[i] = few_key(f, a, i);
    __syncthreads();
    const uint32_t mine = key[token];
    if (!counts(a, mine)) return;
    // Each wave looks through a quarter of the tokens.
    const uint32_t quarter = (a.n + kOpThreads - 1) / kOpThreads * 64u;
    const uint32_t b = w * quarter, e = min(a.n, b + quarter);
    uint32_t n = 0, before = 0;
    for (uint32_t i = b + lane; i - lane < e; i += 64u) {
        const bool same = i < e && key[i] == mine;
        n += (uint32_t)__popcll(__ballot(same));
        before |= __ballot(same && i < token) != 0;
    }
    if (lane == 0) found[w] = n, earlier[w] = before;
    __syncthreads();
    uint32_t at = 0, all = 0, first = 0;
#pragma unroll
    for (uint32_t i = 0; i < kWaves; ++i) {
        at += i < w ? found[i] : 0u;
        all += found[i];
        first |= earlier[i];
    }
    if (first) return;  // the first token of the id adds this one's row
    for (uint32_t i = b + lane; i - lane < e; i += 64u) {
        const bool same = i < e && key[i] == mine;
        const uint64_t votes = __ballot(same);
        if (same) list[at + (uint32_t)__popcll(votes & ((1ull << lane) - 1ull))] = i;
        at += (uint32_t)__popcll(votes);
    }
    __syncthreads();
    const bool whole = u < a.pieces, here = u < a.units;
    const size_t col = whole ? (size_t)u * P::N : (size_t)a.pieces * P::N + (u - a.pieces);
    const uint32_t share = (all + kWaves - 1) / kWaves, end = min(all, (w + 1) * share);
    typename P::f32 acc = 0.0f;
    for (uint32_t i0 = w * share; i0 < end; i0 += kRowsAtOnce) {
        typename P::vec v[kRowsAtOnce];
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r) {
            v[r] = (typename P::vec)(T)0.0f;
            if (!here || i0 + r >= end) continue;
            const T *src = dout + (int64_t)list[i0 + r] * a.ds + col;
            if (whole) v[r] = load_piece<true>(src);
            else v[r][0] = *src;
        }
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r) acc += widen<T>(v[r]);
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w || !here) return;
#pragma unroll
    for (uint32_t i = 1; i < kWaves; ++i) acc += part[i][lane];
    O *dst = table + (int64_t)mine * a.ts + col;
    if (whole) put_piece<T>(dst, acc, a);
    else put(dst, acc[0], a);
}

size_t round_up(size_t v) { return (v + 255) & ~(size_t)255; }

struct GradPlan {
    size_t sort_bytes, index_bytes, part_bytes, bytes;
    uint32_t chunk, chunks;
    bool few;
};

GradPlan grad_plan(int64_t n, int64_t num_rows, int64_t width) {
    GradPlan p{};
    // About as many workgroups as the device holds at once, against three launches:
    // 300 tokens, 2000 x 300 bf16 4.8 us and 11.3, 1000, 50000 x 1000 21.4 and 22.6, 110,
    // 35742 x 1812 f32 34.0 and 40.5; but 2000, 1000 x 300 18.9 and 12.9, and 100, 130000 x
    // 4000 191 and 175, which the clearing beside the sort writes faster.
    p.few = n <= (int64_t)kFewTokens && n * ((width + 511) / 512) <= 2 * (int64_t)kFewTokens &&
            num_rows * width < (int64_t)1 << 28;
    if (p.few) return p;
    // Long chunks leave few partial rows; shorter ones make two workgroups for every
    // CU where there are few tokens.
    const int64_t cols = (width + 2047) / 2048;
    p.chunk = kMaxChunk;
    while (p.chunk > 8 && n * cols / p.chunk < 512) p.chunk /= 2;
    p.chunks = (uint32_t)((n + p.chunk - 1) / p.chunk);
    p.sort_bytes = round_up(sort_workspace(n, num_rows));
    p.index_bytes = round_up((size_t)n * 4);
    p.part_bytes = p.chunks > 1 ? (size_t)p.chunks * 2 * (size_t)width * 4 : 0;
    p.bytes = p.sort_bytes + 2 * p.index_bytes + p.part_bytes;
    return p;
}

template <class T, class O>
hipError_t queue_grad(const segtopk_rows *dout, const segtopk_rows *dtable, const GradArgs &a,
                      hipStream_t stream) {
    if (!a.chunks) return hipSuccess;  // no tokens: nothing to add, and dout may be absent
    O *table = static_cast<O *>(dtable->data);
    const hipError_t err = launch(sum_kernel<T, O>, dim3(a.chunks * a.cols), kOpThreads, stream, 0,
                                  static_cast<const T *>(dout->data), table, a);
    if (err != hipSuccess || a.chunks < 2) return err;
    const int64_t y = (a.width + 255) / 256;
    return launch(finish_kernel<O>, dim3(a.chunks - 1, (unsigned)(y < 64 ? y : 64)), kOpThreads,
                  stream, 0, table, a);
}

template <class T, class O>
hipError_t queue_few(const segtopk_rows *dout, const segtopk_rows *dtable, const GradArgs &a,
                     FewArgs f, hipStream_t stream) {
    f.cols = (a.units + 63u) / 64u;
    f.sums = a.n * f.cols;
    const int64_t fit = 16384 / (a.width * (int64_t)sizeof(O));
    f.rows = fit < 1 ? 1u : fit < (int64_t)kFewRows ? (uint32_t)fit : kFewRows;
    int64_t clears = a.accumulate ? 0 : (a.num_rows + (int64_t)f.rows - 1) / f.rows;
    if (clears > kFillBlocks) clears = kFillBlocks;
    if (!(f.sums + clears)) return hipSuccess;
    return launch(few_kernel<T, O>, dim3(f.sums + (uint32_t)clears), kOpThreads, stream, 0,
                  static_cast<const T *>(a.n ? dout->data : nullptr), static_cast<O *>(dtable->data),
                  a, f);
}

bool good_sizes(int64_t n, int64_t num_rows, int64_t width) {
    return n >= 0 && n <= INT32_MAX && num_rows >= 0 && num_rows < INT32_MAX && width >= 1 &&
           width <= INT32_MAX;
}

}  // namespace
}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int64_t segtopk_embedding_backward_workspace(int64_t n, int64_t num_rows,
                                                        int64_t width) {
    if (!good_sizes(n, num_rows, width)) return 0;
    return (int64_t)grad_plan(n, num_rows, width).bytes;
}

extern "C" int segtopk_embedding_backward(const segtopk_rows *dout, const segtopk_rows *dtable,
                                          const void *ids, int32_t id_type, int64_t n,
                                          int64_t num_rows, int64_t width, float scale,
                                          int64_t padding_id, int32_t accumulate, void *workspace,
                                          int64_t workspace_bytes, hipStream_t stream) {
    const int ib = index_bytes(id_type);
    if (!ib || !good_sizes(n, num_rows, width)) return SEGTOPK_INVALID_ARGUMENT;
    if (num_rows == 0) return SEGTOPK_OK;
    if (!good_rows(dtable, width)) return SEGTOPK_INVALID_ARGUMENT;
    if (n && (!ids || !aligned(ids, ib) || !good_rows(dout, width) ||
              (dtable->type != dout->type && dtable->type != SEGTOPK_KEY_F32)))
        return SEGTOPK_INVALID_ARGUMENT;
    const GradPlan p = grad_plan(n, num_rows, width);
    const int64_t per = 16 / element_bytes(n ? dout->type : dtable->type);
    const int64_t units = width / per + width % per, cols = (units + kOpThreads - 1) / kOpThreads;
    // A launch holds fewer than 2^32 threads.
    if ((int64_t)p.chunks * cols >= (1 << 24) - 1) return SEGTOPK_NOT_SUPPORTED;
    if (p.bytes && (!workspace || !aligned(workspace, 256))) return SEGTOPK_INVALID_ARGUMENT;
    if (workspace_bytes < 0 || (size_t)workspace_bytes < p.bytes) return SEGTOPK_SCRATCH_TOO_SMALL;

    GradArgs a{};
    a.n = (uint32_t)n;
    a.chunk = p.chunk;
    a.chunks = p.chunks;
    a.num_rows = (uint32_t)num_rows;
    a.padding = padding_id >= 0 && padding_id < num_rows ? (uint32_t)padding_id : 0xFFFFFFFFu;
    a.pieces = (uint32_t)(width / per);
    a.units = (uint32_t)units;
    a.cols = (uint32_t)cols;
    a.scale = scale;
    a.accumulate = accumulate != 0;
    a.width = width;
    a.ds = n ? dout->stride : 0;
    a.ts = dtable->stride;
    // Calls f with a value of dout's element type and one of the table's.
    const auto by_types = [&](auto f) {
        return with_type(n ? dout->type : dtable->type, [&](auto t) {
            return status(dtable->type == SEGTOPK_KEY_F32 ? f(t, float{}) : f(t, t));
        });
    };
    if (p.few)
        return by_types([&](auto t, auto o) {
            return queue_few<decltype(t), decltype(o)>(
                dout, dtable, a, FewArgs{ids, id_type == SEGTOPK_KEY_I64}, stream);
        });

    char *ws = static_cast<char *>(workspace);
    int32_t *order = reinterpret_cast<int32_t *>(ws + p.sort_bytes);
    uint32_t *sorted = reinterpret_cast<uint32_t *>(ws + p.sort_bytes + p.index_bytes);
    a.order = order;
    a.sorted = sorted;
    a.part = reinterpret_cast<float *>(ws + p.sort_bytes + 2 * p.index_bytes);
    // A table in one piece is cleared beside the sort, before it is known which of
    // its rows are used: at most one more row is written for each of dout's.
    const int64_t table_bytes = num_rows * width * element_bytes(dtable->type);
    const bool flat = (dtable->stride == width || num_rows == 1) && aligned(dtable->data, 16);
    const Fill fill{dtable->data, flat && !accumulate ? (uint64_t)table_bytes : 0,
                    streams(table_bytes)};
    if (!flat && !accumulate) {
        const unsigned grid = (unsigned)(num_rows < kFillBlocks ? num_rows : kFillBlocks);
        const int st = with_type(dtable->type, [&](auto o) {
            using O = decltype(o);
            return status(launch(clear_kernel<O>, dim3(grid), kOpThreads, stream, 0,
                                 static_cast<O *>(dtable->data), (uint32_t)num_rows, width,
                                 dtable->stride));
        });
        if (st != SEGTOPK_OK) return st;
    }
    if (queue_sort(ids, id_type, n, num_rows, order, nullptr, nullptr, sorted, workspace, stream,
                   &fill) != hipSuccess)
        return SEGTOPK_HIP_ERROR;
    return by_types([&](auto t, auto o) {
        return queue_grad<decltype(t), decltype(o)>(dout, dtable, a, stream);
    });
}
