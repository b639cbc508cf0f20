// quantize.hip -- rows, matrices and transposed rows in 8 bits, with a scale for
// each block of 128.
//
//   a = max |x| over the block, at least 2^-96
//   scale = a / 448,   q = e4m3(x * (448 / a))
// each operation rounded once to nearest even, so that the same numbers come from
// any program that follows the definition.  |x| (448 / a) rounds to 448 at most, so
// nothing saturates.  The maximum is taken of the magnitudes' bits, which order as
// the magnitudes do and keep inf and NaN: they make the block's scale inf or NaN.
//
// Bound by memory: 16 lanes hold a block of a row, 8 elements each, and write 8
// bytes a lane; a token is read once for all of its slots.  65536 rows of 4096 in bf16
// 139 us, 5.8 TB/s; 8192 tokens of 4096 to 8 slots each 60 us, 5.7; 128 matrices of 2048 x
// 4096 588 us, 5.5.  Transposed, 65536 rows of 2048 and 4096 columns 275 us, 4.4: the vector
// units are busy 59% of that, and what is written goes to as many places as there are columns.
#include "quantize.h"

namespace segtopk_ops {
namespace {

constexpr float kMost = 448.0f;
constexpr uint32_t kLeast = 0x0F800000u;  // the bits of 2^-96

// Four values in 8 bits.
__device__ inline uint32_t pack4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
__device__ inline uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ inline uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// 8 elements from an unaligned place.
template <class T> __device__ inline void load8(const T *p, float *x) {
    typedef T mem __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    const mem v = *reinterpret_cast<const mem *>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (float)v[j];
}
template <class T>
__device__ inline void load8_of(const T *p, uint32_t have, float *x) {
    if (have >= 8) {
        load8(p, x);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (uint32_t)j < have ? (float)p[j] : 0.0f;
}

struct RowsArgs {
    int64_t stride, qstride;
    uint8_t *q;
    float *scales;
    const int32_t *position;
    const int64_t *kept;
    uint32_t tokens, k, width, blocks;
};

constexpr uint32_t kRowBlocks = kOpThreads / 16;  // blocks of a workgroup

template <class T>
__global__ __launch_bounds__(kOpThreads) void quantize_rows_kernel(const T *x, RowsArgs a) {
    const uint32_t unit = blockIdx.x * kRowBlocks + threadIdx.x / 16;  // below 2^28
    if (unit >= a.tokens * a.blocks) return;                           // 16 lanes at once
    const uint32_t token = unit / a.blocks, block = unit % a.blocks;
    const uint32_t lane = threadIdx.x % 16, at = block * 128 + lane * 8;
    const uint32_t have = at < a.width ? a.width - at : 0u;
    float v[8];
    load8_of(x + (int64_t)token * a.stride + at, have, v);
    uint32_t m = kLeast;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = larger(m, magnitude(v[j]));
    m = join<16>(m, [](uint32_t p, uint32_t q) { return larger(p, q); });
    const float most = __uint_as_float(m), inverse = kMost / most, scale = most / kMost;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inverse;
    const uint2 bits{pack4(v[0], v[1], v[2], v[3]), pack4(v[4], v[5], v[6], v[7])};
    const bool writes = at < ((a.width + 15u) & ~15u);
    if (!a.position) {
        if (writes) *reinterpret_cast<uint2 *>(a.q + (int64_t)token * a.qstride + at) = bits;
        if (lane == 0) a.scales[(int64_t)token * a.blocks + block] = scale;
        return;
    }
    // The places of 16 slots at once, one to a lane: loads between the stores would each be waited
    // for (8192 tokens of 4096 in bf16, 8 slots each: 68 -> 60 us).
    const int64_t slots = (int64_t)a.tokens * a.k, kept = a.kept ? *a.kept : slots;
    for (uint32_t j0 = 0; j0 < a.k; j0 += 16) {
        const int32_t own = j0 + lane < a.k ? a.position[(int64_t)token * a.k + j0 + lane] : -1;
        for (uint32_t j = 0; j < 16 && j0 + j < a.k; ++j) {
            const int64_t p = __shfl(own, (int)j, 16);
            if (p < 0 || p >= slots) continue;
            const bool keep = p < kept;
            if (writes)
                *reinterpret_cast<uint2 *>(a.q + p * a.qstride + at) = keep ? bits : uint2{0u, 0u};
            if (lane == 0) a.scales[p * a.blocks + block] = keep ? scale : 0.0f;
        }
    }
}

struct BlocksArgs {
    int64_t matrix_stride, stride, qmatrix_stride, qstride;
    uint8_t *q;
    float *scales;
    uint32_t rows, width, row_blocks, col_blocks;
};

// A workgroup a block of 128 x 128, held in registers.
template <class T>
__global__ __launch_bounds__(kOpThreads) void quantize_blocks_kernel(const T *x, BlocksArgs a) {
    __shared__ uint32_t part[kOpThreads / 64];
    const uint32_t cb = blockIdx.x % a.col_blocks, rest = blockIdx.x / a.col_blocks;
    const uint32_t rb = rest % a.row_blocks, e = rest / a.row_blocks;
    const uint32_t at = cb * 128 + threadIdx.x % 16 * 8, row0 = rb * 128 + threadIdx.x / 16;
    const uint32_t have = at < a.width ? a.width - at : 0u;
    const T *m0 = x + (int64_t)e * a.matrix_stride;
    float v[8][8];
    uint32_t m = kLeast;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t r = row0 + i * 16;
        load8_of(m0 + (int64_t)r * a.stride + at, r < a.rows ? have : 0u, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = larger(m, magnitude(v[i][j]));
#pragma unroll
    for (int d = 32; d; d >>= 1) m = larger(m, __shfl_xor(m, d));
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kOpThreads / 64; ++w) m = larger(m, part[w]);
    const float most = __uint_as_float(m), inverse = kMost / most;
    uint8_t *q0 = a.q + (int64_t)e * a.qmatrix_stride;
    const bool writes = at < ((a.width + 15u) & ~15u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t r = row0 + i * 16;
        if (r >= a.rows || !writes) continue;
        float *f = v[i];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= inverse;
        *reinterpret_cast<uint2 *>(q0 + (int64_t)r * a.qstride + at) =
            uint2{pack4(f[0], f[1], f[2], f[3]), pack4(f[4], f[5], f[6], f[7])};
    }
    if (threadIdx.x == 0) a.scales[blockIdx.x] = most / kMost;
}

// A workgroup 128 rows of an expert by 64 columns: each thread 4 neighbouring rows
// of 8 columns, so that a column's four values are one word of the transposed
// tile, which is written from LDS in pieces of 16 bytes.
constexpr uint32_t kTurnCols = 64;

template <class T>
__global__ __launch_bounds__(kOpThreads) void quantize_turned_kernel(const T *one, int64_t one_stride,
                                                                     Turned one_turned, const T *two,
                                                                     int64_t two_stride,
                                                                     Turned two_turned, Segments seg) {
    __shared__ __attribute__((aligned(16))) uint32_t part[kOpThreads / 16][kTurnCols];
    __shared__ __attribute__((aligned(16))) float factor[kTurnCols];
    __shared__ __attribute__((aligned(16))) uint8_t tile[kTurnCols * 128];
    const uint32_t ones = (one_turned.width + kTurnCols - 1) / kTurnCols;
    const uint32_t cols = ones + (two_turned.width + kTurnCols - 1) / kTurnCols;
    const uint32_t b = blockIdx.x / cols, group = blockIdx.x % cols;
    const bool first = group < ones;
    const T *x = first ? one : two;
    const int64_t stride = first ? one_stride : two_stride;
    const Turned t = first ? one_turned : two_turned;
    const uint32_t c0 = (first ? group : group - ones) * kTurnCols;
    Cursor cursor{0, 0};
    const Tile mine = find_tile(seg, b, 128, 1, cursor);
    if (mine.expert >= seg.experts) return;
    const uint32_t i = threadIdx.x, col = i % 8 * 8, row = i / 8 * 4;
    const uint32_t have = c0 + col < t.width ? t.width - c0 - col : 0u;
    float v[4][8];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t at = mine.begin + row + r;
        load8_of(x + at * stride + c0 + col, at < mine.end ? have : 0u, v[r]);
    }
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = kLeast;
#pragma unroll
        for (int r = 0; r < 4; ++r) m[j] = larger(m[j], magnitude(v[r][j]));
        m[j] = larger(m[j], __builtin_amdgcn_update_dpp(m[j], m[j], 0x128, 0xF, 0xF, false));  // 8 lanes on
    }
    if (i % 16 < 8) {
        uint4 *to = reinterpret_cast<uint4 *>(&part[i / 16][col]);
        to[0] = uint4{m[0], m[1], m[2], m[3]};
        to[1] = uint4{m[4], m[5], m[6], m[7]};
    }
    __syncthreads();
    if (i < kTurnCols) {
        uint32_t most = kLeast;
#pragma unroll
        for (uint32_t w = 0; w < kOpThreads / 16; ++w) most = larger(most, part[w][i]);
        factor[i] = kMost / __uint_as_float(most);
        if (c0 + i < t.width) t.scales[(int64_t)b * t.width + c0 + i] = __uint_as_float(most) / kMost;
    }
    __syncthreads();
    // Column c's 16-byte piece p is at piece p ^ (c / 8): neighbouring lanes write neighbouring
    // columns' groups, and each piece meets other banks.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float f = factor[col + j];
        *reinterpret_cast<uint32_t *>(tile + (col + j) * 128 + (((row / 16) ^ (col / 8)) * 16 + row % 16)) =
            pack4(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f);
    }
    __syncthreads();
    for (uint32_t p = i; p < kTurnCols * 8; p += kOpThreads) {
        const uint32_t c = p / 8, piece = p % 8;
        if (c0 + c < t.width)
            *reinterpret_cast<uint4 *>(t.q + (int64_t)(c0 + c) * t.stride + (int64_t)b * 128 + piece * 16) =
                *reinterpret_cast<const uint4 *>(tile + c * 128 + (piece ^ (c / 8)) * 16);
    }
}

bool good_matrices(const segtopk_matrices *m, int64_t matrices, int64_t rows, int64_t width) {
    const int b = m ? element_bytes(m->type) : 0;
    return b && m->data && aligned(m->data, b) && m->stride >= width && m->matrix_stride >= 0 &&
           matrices >= 0 && rows >= 0;
}

}  // namespace

int queue_quantize_turned(const segtopk_rows &one, const Turned &one_turned, const segtopk_rows &two,
                          const Turned &two_turned, const Segments &seg, hipStream_t stream) {
    const int64_t cols = ((int64_t)one_turned.width + kTurnCols - 1) / kTurnCols +
                         ((int64_t)two_turned.width + kTurnCols - 1) / kTurnCols;
    if (cols * (int64_t)seg.tiles_most > kMostBlocks) return SEGTOPK_NOT_SUPPORTED;
    return with_type(one.type, [&](auto v) {
        using T = decltype(v);
        return status(launch(quantize_turned_kernel<T>, dim3((unsigned)(cols * seg.tiles_most)),
                             kOpThreads, stream, 0, static_cast<const T *>(one.data), one.stride,
                             one_turned, static_cast<const T *>(two.data), two.stride, two_turned,
                             seg));
    });
}

}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int segtopk_quantize_rows(const segtopk_rows *x, const segtopk_rows *q, float *scales,
                                     int64_t tokens, int64_t k, int64_t width,
                                     const int32_t *position, const int64_t *kept,
                                     hipStream_t stream) {
    if (tokens < 0 || k < 1 || width < 1 || width >= INT32_MAX - 128 || tokens > INT32_MAX / k)
        return SEGTOPK_INVALID_ARGUMENT;
    if (!tokens) return SEGTOPK_OK;
    if ((!position && (k != 1 || kept)) ||
        !good_rows(x, width) || !good_rows8(q, width) || !scales || !aligned(scales, 4) ||
        (position && !aligned(position, 4)) || (kept && !aligned(kept, 8)))
        return SEGTOPK_INVALID_ARGUMENT;
    RowsArgs a{x->stride, q->stride, static_cast<uint8_t *>(q->data), scales, position, kept,
               (uint32_t)tokens, (uint32_t)k, (uint32_t)width, (uint32_t)((width + 127) / 128)};
    const int64_t groups = (tokens * a.blocks + kRowBlocks - 1) / kRowBlocks;
    if (groups > kMostBlocks) return SEGTOPK_NOT_SUPPORTED;
    return with_type(x->type, [&](auto v) {
        using T = decltype(v);
        return status(launch(quantize_rows_kernel<T>, dim3((unsigned)groups), kOpThreads, stream, 0,
                             static_cast<const T *>(x->data), a));
    });
}

extern "C" int segtopk_quantize_blocks(const segtopk_matrices *x, const segtopk_matrices *q,
                                       float *scales, int64_t matrices, int64_t rows, int64_t width,
                                       hipStream_t stream) {
    if (matrices < 0 || rows < 0 || width < 1 || matrices >= INT32_MAX || rows >= INT32_MAX - 128 ||
        width >= INT32_MAX - 128)
        return SEGTOPK_INVALID_ARGUMENT;
    if (!matrices || !rows) return SEGTOPK_OK;
    if (!good_matrices(x, matrices, rows, width) || !good_matrices8(q, width) || !scales ||
        !aligned(scales, 4))
        return SEGTOPK_INVALID_ARGUMENT;
    BlocksArgs a{x->matrix_stride, x->stride, q->matrix_stride, q->stride,
                 static_cast<uint8_t *>(q->data), scales, (uint32_t)rows, (uint32_t)width,
                 (uint32_t)((rows + 127) / 128), (uint32_t)((width + 127) / 128)};
    const int64_t each = (int64_t)a.row_blocks * a.col_blocks;
    if (each > kMostBlocks / matrices) return SEGTOPK_NOT_SUPPORTED;
    return with_type(x->type, [&](auto v) {
        using T = decltype(v);
        return status(launch(quantize_blocks_kernel<T>, dim3((unsigned)(each * matrices)),
                             kOpThreads, stream, 0, static_cast<const T *>(x->data), a));
    });
}
