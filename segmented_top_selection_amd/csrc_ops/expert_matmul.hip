// expert_matmul.hip -- the experts' products in 8 bits with a scale for each block
// of 128, and the gradient of their weights.
//
//   out[r][n] = sum_b sx[r][b] sw[n / 128][b] sum_{c in block b} qx[r][c] qw[n][c]
//
// One matrix instruction (16 x 16 x 128) does the inner sum of a block for 16 x 16
// results; its four sums a lane are multiplied by the block's scales and added up in
// 32 bits.
//
// The 8-bit instruction adds up 8 products at a time with the smaller ones cut off
// 2^-13 below the largest (the exponents' sum): 1.5e-5 of a sum of random values,
// far below the 2^-9 and 2^-12 that a result in bf16 or f16 is rounded by, and taken
// there for its rate, 4500 TFLOP/s against 1900.  A result in 32 bits is held to them:
// its operands are widened to bf16, which holds e4m3 whole, and multiplied by the
// bf16 instruction, whose sums are right to 32 bits.
//
// The operand whose index is the result's fast one ("columns": n) is the
// instruction's first, so that a lane holds neighbouring columns of one row: it
// needs one scale a row tile, and stores pieces of a row.
#include <type_traits>

#include "quantize.h"

namespace segtopk_ops {
namespace {

typedef int Frag __attribute__((ext_vector_type(8)));
typedef int Quarter __attribute__((ext_vector_type(4)));
typedef float Sums __attribute__((ext_vector_type(4)));

struct MulArgs {
    const uint8_t *rows, *cols;  // both with what is summed over contiguous
    int64_t row_stride, col_stride, col_matrix;
    const float *row_scales, *col_scales;
    void *out;
    int64_t out_stride, out_matrix;
    Segments seg;
    uint32_t width, depth;  // of the product: columns, and what is summed over
    uint32_t height;        // rows of each matrix (the weights' gradient)
    uint32_t col_tiles, row_tiles;
    uint32_t accumulate;
};

typedef __bf16 Wide __attribute__((ext_vector_type(8)));
typedef __bf16 Pair __attribute__((ext_vector_type(2)));

// 16 x 128 of an operand as the instruction takes it; EXACT: as bf16, four times 32
// columns.
template <bool EXACT> struct Operand {
    Frag v;
};
template <> struct Operand<true> {
    Wide v[4];
};

__device__ inline Wide widen8(int lo, int hi) {
    const Pair a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const Pair b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const Pair c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const Pair d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return Wide{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
template <bool EXACT> __device__ inline Operand<EXACT> operand(Frag f) {
    if constexpr (EXACT)
        return {{widen8(f[0], f[1]), widen8(f[2], f[3]), widen8(f[4], f[5]), widen8(f[6], f[7])}};
    else return {f};
}

template <bool EXACT>
__device__ inline Sums multiply(const Operand<EXACT> &a, const Operand<EXACT> &b) {
    Sums s{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (EXACT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], s, 0, 0, 0);
        return s;
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, s, 0, 0, 0, 0, 0, 0);
    }
}

typedef __attribute__((address_space(3))) void *LdsPtr;
typedef const __attribute__((address_space(1))) void *GlobalPtr;
template <int BYTES> __device__ inline void to_lds(const void *from, void *to) {
    static_assert(BYTES == 4 || BYTES == 16, "");
    if constexpr (BYTES == 16) __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)to, 16, 0, 0);
    else __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)to, 4, 0, 0);
}

// Waits until at most N of the wave's loads are under way.
template <int N> __device__ inline void loads_left() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x70 | 0xF00);
}

// Where the tile in LDS holds piece c of row r: rows are 128 bytes, and a row's 8
// pieces are swapped so that the lanes that read one piece of several rows meet
// different banks.  Lanes 4 apart read columns 4 * NT apart.
template <int NT> __device__ inline uint32_t swap_of(uint32_t r) {
    return NT == 1 ? r & 7u : (r ^ ((r / NT) & 4u)) & 7u;
}

// ROWS x 128 bytes of an operand into LDS, 8 rows to an instruction of a wave.
template <int ROWS, int WAVES, int NT>
__device__ inline void load_tile(const uint8_t *from, int64_t stride, uint32_t last, uint32_t k0,
                                 uint32_t depth, uint8_t *to) {
    const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
#pragma unroll
    for (int i = 0; i < ROWS / 8 / WAVES; ++i) {
        const uint32_t r0 = (i * WAVES + wave) * 8, r = r0 + lane / 8;
        uint32_t at = k0 + ((lane % 8) ^ swap_of<NT>(r)) * 16;
        if (at >= depth) at = 0;  // past the row's end: anything
        to_lds<16>(from + (int64_t)(r < last ? r : last) * stride + at, to + r0 * 128);
    }
}

// Zeros from byte `have` on of each row.
template <int ROWS, int THREADS, int NT>
__device__ inline void clear_tail(uint8_t *tile, uint32_t have) {
    for (uint32_t u = threadIdx.x; u < ROWS * 8; u += THREADS) {
        const uint32_t r = u / 8, c = u % 8;
        if (c * 16 + 16 <= have) continue;
        Quarter *p = reinterpret_cast<Quarter *>(tile + r * 128 + (c ^ swap_of<NT>(r)) * 16);
        Quarter v = *p;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int b = (int)have - (int)(c * 16 + w * 4);
            v[w] &= b >= 4 ? -1 : b <= 0 ? 0 : (int)((1u << (b * 8)) - 1u);
        }
        *p = v;
    }
}

__device__ inline Frag fragment(const uint8_t *row, uint32_t swap) {
    const uint32_t g = threadIdx.x % 64 / 16;
    const Quarter a = *reinterpret_cast<const Quarter *>(row + (g ^ swap) * 16);
    const Quarter b = *reinterpret_cast<const Quarter *>(row + ((g + 4) ^ swap) * 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// N neighbouring results.
template <class T, int N>
__device__ inline void store(T *p, const float *v, uint32_t have, bool accumulate) {
    typedef T mem __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    if (have >= (uint32_t)N) {
        mem m;
        if (accumulate) {
            m = *reinterpret_cast<mem *>(p);
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = (T)((float)m[i] + v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = (T)v[i];
        }
        *reinterpret_cast<mem *>(p) = m;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((uint32_t)i < have) p[i] = (T)((accumulate ? (float)p[i] : 0.0f) + v[i]);
    }
}

// BM rows by BN columns, by WM x WN waves.  TURNED: the weights' gradient, where both
// operands are transposed, have a scale for each index, and are summed over the
// tiles of an expert.
template <class T, int BM, int BN, int WM, int WN, bool TURNED>
__global__ __launch_bounds__(WM *WN * 64) void product_kernel(MulArgs a) {
    constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    constexpr int kLoads = (BM + BN) / 8 / kWaves;
    constexpr bool kExact = std::is_same<T, float>::value;
    __shared__ __attribute__((aligned(16))) uint8_t row_tile[2][BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t col_tile[2][BN * 128];
    __shared__ __attribute__((aligned(16))) float row_scale[2][BM];
    __shared__ __attribute__((aligned(16))) float col_scale[2][TURNED ? BN : 4];

    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t wm = wave % WM, wn = wave / WM;
    uint32_t blocks, k_first = 0, row0, expert, have_rows;
    int64_t first_row = 0;
    const uint32_t n0 = blockIdx.x % a.col_tiles * BN;
    if constexpr (TURNED) {
        const uint32_t rest = blockIdx.x / a.col_tiles;
        row0 = rest % a.row_tiles * BM;
        expert = rest / a.row_tiles;
        // The expert's tiles of 128, and those before it.
        uint32_t before = 0, own = 0;
        for (uint32_t e0 = 0; e0 <= expert; e0 += 64) {
            const uint32_t e = e0 + lane;
            uint32_t n = 0;
            if (e <= expert) {
                const int64_t b = cut_offset(a.seg, e), end = cut_offset(a.seg, e + 1);
                n = end > b ? (uint32_t)((end - b + 127) / 128) : 0u;
            }
            own = __shfl(n, (int)(expert & 63u));
            if (e < expert) before += n;
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) before += __shfl_xor(before, d);
        before = before < a.seg.tiles_most ? before : a.seg.tiles_most;
        own = own < a.seg.tiles_most - before ? own : a.seg.tiles_most - before;
        k_first = before * 128;
        blocks = own;
        have_rows = a.height - row0;
    } else {
        const Tile t = find_tile(a.seg, blockIdx.x / a.col_tiles, BM);
        expert = t.expert;
        row0 = 0;
        first_row = t.begin;
        if (expert >= a.seg.experts) return;
        have_rows = (uint32_t)(t.end - t.begin < BM ? t.end - t.begin : BM);
        blocks = (a.depth + 127) / 128;
    }
    expert = __builtin_amdgcn_readfirstlane(expert);
    blocks = __builtin_amdgcn_readfirstlane(blocks);
    const uint32_t last_row = (have_rows < BM ? have_rows : BM) - 1;
    const uint32_t last_col = (a.width - n0 < BN ? a.width - n0 : BN) - 1;
    const uint8_t *rows = a.rows + (TURNED ? (int64_t)row0 : first_row) * a.row_stride + k_first;
    const uint8_t *cols = a.cols + (TURNED ? (int64_t)0 : (int64_t)expert * a.col_matrix) +
                          (int64_t)n0 * a.col_stride + k_first;
    const uint32_t depth_blocks = (a.depth + 127) / 128;
    const uint32_t depth = TURNED ? blocks * 128 : a.depth;

    Sums acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Sums{0.0f, 0.0f, 0.0f, 0.0f};

    const auto load = [&](uint32_t b, int s) {
        load_tile<BM, kWaves, 1>(rows, a.row_stride, last_row, b * 128, depth, row_tile[s]);
        load_tile<BN, kWaves, NT>(cols, a.col_stride, last_col, b * 128, depth, col_tile[s]);
        const uint32_t part = wave % ((BM + 63) / 64) * 64;
        const uint32_t r = part + lane < last_row ? part + lane : last_row;
        if constexpr (TURNED) {
            to_lds<4>(a.row_scales + (int64_t)(k_first / 128 + b) * a.height + row0 + r,
                      row_scale[s] + part);
            const uint32_t cpart = wave % ((BN + 63) / 64) * 64;
            const uint32_t c = cpart + lane < last_col ? cpart + lane : last_col;
            to_lds<4>(a.col_scales + (int64_t)(k_first / 128 + b) * a.width + n0 + c,
                      col_scale[s] + cpart);
        } else {
            to_lds<4>(a.row_scales + (first_row + r) * depth_blocks + b, row_scale[s] + part);
        }
    };
    const float *sw = nullptr;  // of the wave's columns
    if constexpr (!TURNED) {
        uint32_t nb = (n0 + wn * NT * 16) / 128;
        const uint32_t most = (a.width - 1) / 128;
        nb = __builtin_amdgcn_readfirstlane(nb < most ? nb : most);
        sw = a.col_scales + ((int64_t)expert * (most + 1) + nb) * depth_blocks;
    }

    const auto compute = [&](uint32_t b, int s) {
        const uint32_t l = lane % 16;
        const float cs = TURNED ? 1.0f : sw[b];
        Operand<kExact> c[NT];
        Sums cscale[TURNED ? NT : 1];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t n = wn * NT * 16 + l / 4 * (4 * NT) + j * 4 + l % 4;
            c[j] = operand<kExact>(fragment(col_tile[s] + n * 128, swap_of<NT>(n)));
            if constexpr (TURNED)
                cscale[j] = *reinterpret_cast<const Sums *>(
                    &col_scale[s][wn * NT * 16 + lane / 16 * (4 * NT) + j * 4]);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint32_t m = (wm * MT + i) * 16 + l;
            const Operand<kExact> r =
                operand<kExact>(fragment(row_tile[s] + m * 128, swap_of<1>(m)));
            const float scale = row_scale[s][m] * cs;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const Sums p = multiply<kExact>(c[j], r);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    acc[i][j][x] = fmaf(p[x], TURNED ? scale * cscale[TURNED ? j : 0][x] : scale,
                                        acc[i][j][x]);
            }
        }
    };

    if (blocks) load(0, 0);
    for (uint32_t b = 0; b < blocks; ++b) {
        const int s = b & 1;
        if (b + 1 < blocks) {
            load(b + 1, s ^ 1);
            loads_left<kLoads + (TURNED ? 2 : 1)>();
        } else {
            loads_left<0>();
        }
        __syncthreads();
        if (b + 1 == blocks && (depth & 127u)) {
            clear_tail<BM, kThreads, 1>(row_tile[s], depth - b * 128);
            clear_tail<BN, kThreads, NT>(col_tile[s], depth - b * 128);
            __syncthreads();
        }
        compute(b, s);
        __syncthreads();
    }

    T *out = static_cast<T *>(a.out) +
             (TURNED ? (int64_t)expert * a.out_matrix + (int64_t)row0 * a.out_stride
                     : first_row * a.out_stride);
    const uint32_t n = n0 + wn * NT * 16 + lane / 16 * (4 * NT);
    const uint32_t have = n < a.width ? a.width - n : 0u;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const uint32_t m = (wm * MT + i) * 16 + lane % 16;
        if (m <= last_row && have) {
            float v[NT * 4];
#pragma unroll
            for (int j = 0; j < NT * 4; ++j) v[j] = acc[i][j / 4][j % 4];
            store<T, NT * 4>(out + (int64_t)m * a.out_stride + n, v, have, TURNED && a.accumulate);
        }
    }
}

// The rows behind the last expert's: zeros.
template <class T>
__global__ __launch_bounds__(kOpThreads) void clear_rows_kernel(MulArgs a) {
    const int64_t first = cut_offset(a.seg, a.seg.experts);
    for (int64_t r = first + blockIdx.x; r < a.seg.rows; r += gridDim.x) {
        T *row = static_cast<T *>(a.out) + r * a.out_stride;
        for (uint32_t n = threadIdx.x; n < a.width; n += kOpThreads) row[n] = (T)0.0f;
    }
}

bool good_sizes(int64_t rows, int64_t experts, int64_t width, int64_t depth) {
    const int64_t most = INT32_MAX - 1024;
    return rows >= 0 && rows < most && experts >= 1 && experts <= 65535 && width >= 1 &&
           width < most && depth >= 1 && depth < most;
}

struct DweightsSpace {
    int64_t tiles, stride;  // of the transposed rows
    int64_t dout, rows, dout_scales, rows_scales, bytes;
};

DweightsSpace space_of(int64_t num_rows, int64_t experts, int64_t width, int64_t depth) {
    DweightsSpace s;
    s.tiles = tiles_most(num_rows, experts, 128);
    s.stride = s.tiles * 128;
    const auto up = [](int64_t n) { return (n + 255) & ~(int64_t)255; };
    s.dout = 0;
    s.rows = s.dout + up(width * s.stride);
    s.dout_scales = s.rows + up(depth * s.stride);
    s.rows_scales = s.dout_scales + up(s.tiles * width * 4);
    s.bytes = s.rows_scales + up(s.tiles * depth * 4);
    return s;
}

}  // namespace
}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int segtopk_expert_matmul(const segtopk_expert_matmul_args *args, hipStream_t stream) {
    if (!args) return SEGTOPK_INVALID_ARGUMENT;
    const segtopk_expert_matmul_args &q = *args;
    if (!good_sizes(q.num_rows, q.num_experts, q.width, q.depth)) return SEGTOPK_INVALID_ARGUMENT;
    if (!q.num_rows) return SEGTOPK_OK;
    if (!good_rows8(&q.rows, q.depth) || !good_matrices8(&q.weights, q.depth) ||
        !good_rows(&q.out, q.width) || !q.row_scales || !aligned(q.row_scales, 4) ||
        !q.weight_scales || !aligned(q.weight_scales, 4) || !q.offsets || !aligned(q.offsets, 8))
        return SEGTOPK_INVALID_ARGUMENT;
    MulArgs a{};
    a.rows = static_cast<const uint8_t *>(q.rows.data);
    a.cols = static_cast<const uint8_t *>(q.weights.data);
    a.row_stride = q.rows.stride;
    a.col_stride = q.weights.stride;
    a.col_matrix = q.weights.matrix_stride;
    a.row_scales = q.row_scales;
    a.col_scales = q.weight_scales;
    a.out = q.out.data;
    a.out_stride = q.out.stride;
    a.seg = {q.offsets, q.num_rows, (uint32_t)q.num_experts, 0};
    a.width = (uint32_t)q.width;
    a.depth = (uint32_t)q.depth;
    return with_type(q.out.type, [&](auto v) -> int {
        using T = decltype(v);
        const auto go = [&](auto bm, auto bn, auto wm, auto wn) -> int {
            constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
            constexpr int WM = decltype(wm)::value, WN = decltype(wn)::value;
            a.col_tiles = (a.width + BN - 1) / BN;
            const int64_t tiles = tiles_most(q.num_rows, q.num_experts, BM);
            if (tiles > kMostBlocks / a.col_tiles) return SEGTOPK_NOT_SUPPORTED;
            if (launch(product_kernel<T, BM, BN, WM, WN, false>,
                       dim3((unsigned)(tiles * a.col_tiles)), WM * WN * 64, stream, 0,
                       a) != hipSuccess)
                return SEGTOPK_HIP_ERROR;
            return status(launch(clear_rows_kernel<T>, dim3(256), kOpThreads, stream, 0, a));
        };
        using std::integral_constant;
        return go(integral_constant<int, 128>{}, integral_constant<int, 128>{},
                  integral_constant<int, 2>{}, integral_constant<int, 2>{});
    });
}

extern "C" int64_t segtopk_expert_dweights_workspace(int64_t num_rows, int64_t num_experts,
                                                     int64_t width, int64_t depth) {
    if (!good_sizes(num_rows, num_experts, width, depth)) return 0;
    return space_of(num_rows, num_experts, width, depth).bytes;
}

extern "C" int segtopk_expert_dweights(const segtopk_expert_dweights_args *args, void *workspace,
                                       int64_t workspace_bytes, hipStream_t stream) {
    if (!args) return SEGTOPK_INVALID_ARGUMENT;
    const segtopk_expert_dweights_args &q = *args;
    if (!good_sizes(q.num_rows, q.num_experts, q.width, q.depth)) return SEGTOPK_INVALID_ARGUMENT;
    if (q.num_rows && (!good_rows(&q.dout, q.width) || !good_rows(&q.rows, q.depth) ||
                       q.rows.type != q.dout.type))
        return SEGTOPK_INVALID_ARGUMENT;
    const segtopk_matrices &d = q.dweights;
    if (!element_bytes(d.type) || !d.data || !aligned(d.data, element_bytes(d.type)) ||
        d.stride < q.depth || d.matrix_stride < 0 ||
        (q.num_rows && d.type != q.dout.type && d.type != SEGTOPK_KEY_F32) || !q.offsets ||
        !aligned(q.offsets, 8))
        return SEGTOPK_INVALID_ARGUMENT;
    const DweightsSpace s = space_of(q.num_rows, q.num_experts, q.width, q.depth);
    if (workspace_bytes < s.bytes) return SEGTOPK_SCRATCH_TOO_SMALL;
    if (s.bytes && (!workspace || !aligned(workspace, 256))) return SEGTOPK_INVALID_ARGUMENT;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const Segments seg{q.offsets, q.num_rows, (uint32_t)q.num_experts, (uint32_t)s.tiles};
    const Turned dout{ws + s.dout, reinterpret_cast<float *>(ws + s.dout_scales), s.stride,
                      (uint32_t)q.width};
    const Turned rows{ws + s.rows, reinterpret_cast<float *>(ws + s.rows_scales), s.stride,
                      (uint32_t)q.depth};
    constexpr int BM = 128, BN = 128;
    MulArgs a{};
    a.rows = dout.q;
    a.cols = rows.q;
    a.row_stride = a.col_stride = s.stride;
    a.row_scales = dout.scales;
    a.col_scales = rows.scales;
    a.out = d.data;
    a.out_stride = d.stride;
    a.out_matrix = d.matrix_stride;
    a.seg = seg;
    a.width = (uint32_t)q.depth;
    a.height = (uint32_t)q.width;
    a.accumulate = q.accumulate != 0;
    a.col_tiles = (a.width + BN - 1) / BN;
    a.row_tiles = (a.height + BM - 1) / BM;
    const int64_t matrix = (int64_t)a.col_tiles * a.row_tiles;
    if (matrix > kMostBlocks / q.num_experts) return SEGTOPK_NOT_SUPPORTED;
    if (s.tiles) {
        int r = queue_quantize_turned(q.dout, dout, seg, stream);
        if (r == SEGTOPK_OK) r = queue_quantize_turned(q.rows, rows, seg, stream);
        if (r != SEGTOPK_OK) return r;
    }
    return with_type(d.type, [&](auto v) {
        using T = decltype(v);
        return status(launch(product_kernel<T, BM, BN, 2, 2, true>,
                             dim3((unsigned)(matrix * q.num_experts)), 256, stream, 0, a));
    });
}
