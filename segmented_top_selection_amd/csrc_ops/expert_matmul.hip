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
// there for its rate: loops of nothing else reach 4870 TFLOP/s against 2080.  A result
// in 32 bits is held to them: its operands are widened to bf16, which holds e4m3 whole,
// and multiplied by the bf16 instruction, whose sums are right to 32 bits.
//
// The operand whose index is the result's fast one ("columns": n) is the
// instruction's first, so that a lane holds neighbouring columns of one row: it
// needs one scale a row tile, and stores pieces of a row.
//
// Measured in bf16, 128 experts of 4096 to 2048 unless said: 512 rows an expert, 8192 tokens'
// 8 slots shared unevenly, 810 us, 1360 TFLOP/s (a fifth of the tiles' rows are nobody's); one
// matrix of 8192 x 8192 and 8192 rows 555 us, 1980.  The matrix units are busy 38% of that at
// the 1.95 GHz that the device keeps under them; a block of 256 x 256 results needs 2060 clocks
// of them, 64 KiB from L2 (23 bytes a clock and CU: 2850) and 192 KiB out of LDS (1540), which
// the two waves of a SIMD overlap in part.  Few rows (64 experts, 8 each): 97 us, 5.5 TB/s of
// weights.  The weights' gradient, 65536 rows: 1260 us behind 275 of quantization, 500 of them
// the 2.1 GB of results.
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

// A descriptor of memory from `base` on, `bytes` of it: loads past them give zeros.
typedef uint32_t Memory __attribute__((ext_vector_type(4)));
__device__ inline Memory memory(const void *base, int64_t bytes) {
    const uint64_t at = (uint64_t)(uintptr_t)base;
    return Memory{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu,
                  bytes < 0xFFFFFFFFll ? (uint32_t)bytes : 0xFFFFFFFFu, 0x00020000u};
}
// BYTES a lane straight into LDS, lane after lane from `to` on; `to` and `at` are the
// wave's.  No register is written but m0, which nothing else here uses.  The kernel waits for these loads itself (meet): seen
// by the compiler, each would be waited for before the next read of LDS.
template <int BYTES>
__device__ inline void to_lds(Memory from, uint32_t lane_at, uint32_t at, uint32_t to) {
    static_assert(BYTES == 4 || BYTES == 16, "");
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                     :: "v"(lane_at), "s"(from), "s"(at), "s"(to) : "memory");
    else
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
                     :: "v"(lane_at), "s"(from), "s"(at), "s"(to) : "memory");
}
__device__ inline uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// Waits until at most N of the wave's loads are under way, and for all of its LDS
// instructions; then for the workgroup.  (The compiler's own barrier waits for all loads.)
template <int N> __device__ inline void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x70);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
__device__ inline uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
// A number that is the same for the whole workgroup, by the scalar cache.
__device__ inline float uniform_float(const float *p) {
    return *(const __attribute__((address_space(4))) float *)(uintptr_t)p;
}

// Where the tile in LDS holds piece c of row r: rows are 128 bytes, and a row's 8
// pieces are swapped so that the lanes that read one piece of several rows meet
// different banks.  Lanes 4 apart read rows 4 * RUN apart.
template <int RUN> __device__ inline uint32_t swap_of(uint32_t r) {
    return RUN == 1 ? r & 7u : (r ^ ((r / RUN) & 4u)) & 7u;
}

// ROWS x 128 bytes of an operand into LDS, 8 rows to an instruction of a wave.
template <int ROWS, int WAVES, int RUN> struct TileLoad {
    static constexpr int N = ROWS / 8 / WAVES;
    uint32_t at[N];  // of the lane's pieces in the first block

    __device__ inline TileLoad(uint32_t stride, uint32_t wave) {
        const uint32_t lane = threadIdx.x % 64;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t r = (i * WAVES + wave) * 8 + lane / 8;
            at[i] = r * stride + ((lane % 8) ^ swap_of<RUN>(r)) * 16;
        }
    }
    __device__ inline void load(Memory from, uint32_t k0, const uint8_t *to, uint32_t wave) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            to_lds<16>(from, at[i], k0, lds_address(to) + (i * WAVES + wave) * 1024);
    }
};

// Zeros from byte `have` on of each row.
template <int ROWS, int THREADS, int RUN>
__device__ inline void clear_tail(uint8_t *tile, uint32_t have) {
    for (uint32_t u = threadIdx.x; u < ROWS * 8; u += THREADS) {
        const uint32_t r = u / 8, c = u % 8;
        if (c * 16 + 16 <= have) continue;
        Quarter *p = reinterpret_cast<Quarter *>(tile + r * 128 + (c ^ swap_of<RUN>(r)) * 16);
        Quarter v = *p;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int b = (int)have - (int)(c * 16 + w * 4);
            v[w] &= b >= 4 ? -1 : b <= 0 ? 0 : (int)((1u << (b * 8)) - 1u);
        }
        *p = v;
    }
}

// 32 bytes of a row: the pieces g and g + 4 of lane group g, which lie 64 bytes apart.
__device__ inline Frag fragment(const uint8_t *first, const uint8_t *second) {
    const Quarter a = *reinterpret_cast<const Quarter *>(first);
    const Quarter b = *reinterpret_cast<const Quarter *>(second);
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

// A tile of results: its expert, first row and column, how many rows there are from its
// first to the expert's (matrix's) last, and the blocks that are summed over.
struct Spot {
    uint32_t expert, row, col, rows, first, blocks;
};

// What a workgroup multiplies for it; all in scalar registers.
struct Work {
    Memory rows, cols, row_scales, col_scales;
    const float *sw;  // the scales of the wave's columns
    int64_t out;      // the tile's first element
    uint32_t blocks, depth, last_row, width;  // `width`: columns from its first to the matrix's last
};

// BM rows by BN columns, by WM x WN waves.  TURNED: the weights' gradient, where both
// operands are transposed, have a scale for each index, and are summed over the
// tiles of an expert.
//
// A workgroup to a CU (as many as LDS allows) takes tiles in turn; the next tile's first
// block is on its way while this one's results are stored.
template <class T, int BM, int BN, int WM, int WN, bool TURNED>
__global__ __launch_bounds__(WM *WN * 64) void product_kernel(MulArgs a) {
    constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    // A lane's results of RUN products are neighbours, 16 bytes of a row, and four lanes' 64.  In
    // f32 a row's results all in one lane, 64 bytes in four stores, take longer: weights' gradient
    // of 60 experts of 336 x 1410, 4662 rows, 68 against 55 us.  In 16 bits (one store or two) 16
    // experts of 2048 x 2048 are alike; 8 bytes a lane lose: 128 experts of 2048 x 4096 1616
    // and 1736.
    constexpr int RUN = sizeof(T) == 4 ? 1 : 2;
    constexpr bool kExact = std::is_same<T, float>::value;
    __shared__ __attribute__((aligned(16))) uint8_t row_tile[2][BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t col_tile[2][BN * 128];
    __shared__ __attribute__((aligned(16))) float row_scale[2][BM];
    __shared__ __attribute__((aligned(16))) float col_scale[2][TURNED ? BN : 4];

    const uint32_t lane = threadIdx.x % 64;
    const uint32_t wave = uniform(threadIdx.x / 64);
    // The waves of one SIMD (0 and 4, say) have different rows: in a tile that is not
    // full all SIMDs keep the same work.
    const uint32_t wm = wave / WN, wn = wave % WN;
    const uint32_t depth_blocks = (a.depth + 127) / 128;
    Cursor cursor{0, 0};
    uint32_t known = UINT32_MAX, known_first = 0, known_blocks = 0;  // the last expert's blocks

    const auto locate = [&](uint32_t at) {
        Spot s;
        if constexpr (TURNED) {
            s.expert = at / (a.col_tiles * a.row_tiles);
            const Place p = place_of(at % (a.col_tiles * a.row_tiles), a.row_tiles, a.col_tiles);
            if (s.expert != known) {
                known = s.expert;
                const Range r = tiles_of(a.seg, known, 128, cursor);
                // Offsets that are no segments may say anything.
                known_first = uniform(r.first < a.seg.tiles_most ? r.first : a.seg.tiles_most);
                const uint32_t count = uniform(r.count), left = a.seg.tiles_most - known_first;
                known_blocks = count < left ? count : left;
            }
            s.first = known_first;
            s.blocks = known_blocks;
            s.row = p.down * BM;
            s.col = p.across * BN;
            s.rows = a.height - s.row;
        } else {
            const Tile t = find_tile(a.seg, at, BM, a.col_tiles, cursor);
            s.expert = uniform(t.expert);
            s.col = uniform(t.column) * BN;
            s.row = uniform((uint32_t)t.begin);  // below 2^31
            s.rows = uniform((uint32_t)t.end) - s.row;
            s.blocks = depth_blocks;
            s.first = 0;
        }
        return s;
    };
    const auto work_of = [&](const Spot &s) {
        Work w;
        w.blocks = s.blocks;
        w.depth = TURNED ? s.blocks * 128 : a.depth;
        w.last_row = (s.rows < BM ? s.rows : BM) - 1;
        w.width = a.width - s.col;
        const uint32_t last_col = (w.width < BN ? w.width : BN) - 1;
        const uint32_t reach = (w.depth + 15) & ~15u;  // of a row, in bytes
        w.rows = memory(a.rows + (int64_t)s.row * a.row_stride + (int64_t)s.first * 128,
                        (int64_t)w.last_row * a.row_stride + reach);
        w.cols = memory(a.cols + (TURNED ? 0 : (int64_t)s.expert * a.col_matrix) +
                            (int64_t)s.col * a.col_stride + (int64_t)s.first * 128,
                        (int64_t)last_col * a.col_stride + reach);
        if constexpr (TURNED) {
            const int64_t behind = (int64_t)w.blocks - 1;
            w.row_scales = memory(a.row_scales + (int64_t)s.first * a.height + s.row,
                                  (behind * a.height + w.last_row + 1) * 4);
            w.col_scales = memory(a.col_scales + (int64_t)s.first * a.width + s.col,
                                  (behind * a.width + last_col + 1) * 4);
            w.sw = nullptr;
            w.out = (int64_t)s.expert * a.out_matrix + (int64_t)s.row * a.out_stride + s.col;
        } else {
            w.row_scales = memory(a.row_scales + (int64_t)s.row * depth_blocks,
                                  (int64_t)(w.last_row + 1) * depth_blocks * 4);
            w.col_scales = w.row_scales;
            const uint32_t most = (a.width - 1) / 128, nb = (s.col + wn * NT * 16) / 128;
            w.sw = a.col_scales +
                   ((int64_t)s.expert * (most + 1) + (nb < most ? nb : most)) * depth_blocks;
            w.out = (int64_t)s.row * a.out_stride + s.col;
        }
        return w;
    };

    const TileLoad<BM, kWaves, 1> row_load((uint32_t)a.row_stride, wave);
    const TileLoad<BN, kWaves, RUN> col_load((uint32_t)a.col_stride, wave);
    // The scales of the rows: 64 of them a wave, some twice.
    const uint32_t part = wave % ((BM + 63) / 64) * 64, cpart = wave % ((BN + 63) / 64) * 64;
    const uint32_t row_scale_at = (part + lane) * (TURNED ? 4 : depth_blocks * 4);
    const uint32_t scale_step = TURNED ? a.height * 4 : 4;
    const auto load_rows = [&](const Work &w, uint32_t b, int s) {
        row_load.load(w.rows, b * 128, row_tile[s], wave);
        to_lds<4>(w.row_scales, row_scale_at, b * scale_step, lds_address(row_scale[s] + part));
        if constexpr (TURNED)
            to_lds<4>(w.col_scales, (cpart + lane) * 4, b * a.width * 4, lds_address(col_scale[s] + cpart));
    };
    const auto load_cols = [&](const Work &w, uint32_t b, int s) {
        col_load.load(w.cols, b * 128, col_tile[s], wave);
    };
    constexpr int kRowLoads = BM / 8 / kWaves + (TURNED ? 2 : 1), kColLoads = BN / 8 / kWaves;
    const auto start = [&](const Work &w) {
        if (!w.blocks) return;
        load_rows(w, 0, 0);
        load_cols(w, 0, 0);
        if (w.blocks > 1) load_cols(w, 1, 1);
    };

    const uint32_t l = lane % 16;
    // Where the lane's pieces begin.  Four columns on, the pieces of a pair change places.
    const uint32_t col0 = wn * NT * 16 + l / 4 * (4 * RUN) + l % 4;
    const uint32_t col_at = col0 * 128 + ((lane / 16) ^ swap_of<RUN>(col0)) * 16;
    const auto col_of = [](int j) { return j / RUN * RUN * 16 + j % RUN * 4; };
    const uint32_t row_at = (wm * MT * 16 + l) * 128 + ((lane / 16) ^ swap_of<1>(l)) * 16;
    const auto col_operand = [&](int j, int s) {
        const uint8_t *at = col_tile[s] + col_of(j) * 128, *one = at + col_at, *two = at + (col_at ^ 64u);
        return operand<kExact>(RUN > 1 && j % 2 ? fragment(two, one) : fragment(one, two));
    };
    const auto row_operand = [&](int i, int s) {
        const uint8_t *at = row_tile[s] + i * 2048;
        return operand<kExact>(fragment(at + row_at, at + (row_at ^ 64u)));
    };
    Sums acc[MT][NT];
    Operand<kExact> c[NT];
    const auto read_cols = [&](int s) {
#pragma unroll
        for (int j = 0; j < NT; ++j) c[j] = col_operand(j, s);
    };

    // Block b.  Its columns are in registers, its rows in LDS; the next block's rows are on
    // their way to the other half of theirs, and the columns of the one after that to the
    // place of this block's.  Before the last row tile all waves wait for the next block's
    // columns, which replace this one's in the registers as they are used.  Each product's
    // sums are added up a product later.
    constexpr int kAhead = 1;
    const auto step = [&](const Work &w, uint32_t b, auto half) {
        constexpr int s = decltype(half)::value;
        const bool mine = wm * MT * 16 <= w.last_row;
        const bool ragged = (w.depth & 127u) != 0;
        const bool one_more = b + 1 < w.blocks, two_more = b + 2 < w.blocks;
        const float cs = TURNED ? 1.0f : uniform_float(w.sw + b);
        if (one_more) load_rows(w, b + 1, s ^ 1);
        if (two_more) load_cols(w, b + 2, s);
        Sums p[kAhead + 1], cscale[TURNED ? NT : 1];
        float scale[MT];
        Operand<kExact> r, next;
        const auto read_scale = [&](int i) { scale[i] = row_scale[s][(wm * MT + i) * 16 + l]; };
        const auto add = [&](int t) {
            const int i = t / NT, j = t % NT;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                acc[i][j][x] = fmaf(p[t % (kAhead + 1)][x],
                                    TURNED ? scale[i] * cscale[TURNED ? j : 0][x] : scale[i],
                                    acc[i][j][x]);
        };
        if (mine) {
            r = row_operand(0, s);
            if constexpr (TURNED)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    cscale[j] = *reinterpret_cast<const Sums *>(
                        &col_scale[s][wn * NT * 16 + lane / 16 * (4 * RUN) + col_of(j)]);
            read_scale(0);
#pragma unroll
            for (int i = 0; i < MT - 1; ++i) {
                next = row_operand(i + 1, s);
                read_scale(i + 1);
                scale[i] *= cs;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int t = i * NT + j;
                    p[t % (kAhead + 1)] = multiply<kExact>(c[j], r);
                    if (t >= kAhead) add(t - kAhead);
                }
                r = next;
            }
        }
        if (one_more) {
            if (two_more) meet<kRowLoads + kColLoads>();
            else meet<kRowLoads>();
            if (ragged && b + 2 == w.blocks) {
                clear_tail<BN, kThreads, RUN>(col_tile[s ^ 1], w.depth - (b + 1) * 128);
                meet<kRowLoads>();
            }
        }
        if (mine) {
            scale[MT - 1] *= cs;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int t = (MT - 1) * NT + j;
                p[t % (kAhead + 1)] = multiply<kExact>(c[j], r);
                c[j] = col_operand(j, s ^ 1);  // behind the last block: anything
                add(t - kAhead);
            }
#pragma unroll
            for (int t = MT * NT - kAhead; t < MT * NT; ++t) add(t);
        }
        if (one_more) {
            if (two_more) meet<kColLoads>();
            else meet<0>();
            if (ragged && b + 2 == w.blocks) {
                clear_tail<BM, kThreads, 1>(row_tile[s ^ 1], w.depth - (b + 1) * 128);
                meet<0>();
            }
        }
    };

    // Workgroups go to the eight XCDs in turn.  Each XCD has a run of neighbouring tiles, so
    // that an expert's operands are in one cache, or two.
    uint32_t all = a.seg.experts * a.col_tiles * a.row_tiles;
    if constexpr (!TURNED) {
        // Offsets that are no segments may say anything.
        const uint32_t count = uniform(count_tiles(a.seg, BM));
        all = (count < a.seg.tiles_most ? count : a.seg.tiles_most) * a.col_tiles;
    }
    const uint32_t each = (all + 7) / 8, begin = blockIdx.x % 8 * each;
    const uint32_t end = begin + each < all ? begin + each : all, turn = gridDim.x / 8;
    uint32_t at = begin + blockIdx.x / 8;
    // Workgroups of large tiles that begin at up to eight different times, 2 us apart, do not
    // all store or all multiply at once (128 experts of 2048 x 4096, 65536 rows: 915 -> 850 us,
    // their weights' gradient 1649 -> 1595 us).  A start of 13 us later pays for some tiles each.
    if (BM * BN == 65536 && each >= 4 * turn)
        for (uint32_t i = blockIdx.x / 8 % 8; i; --i) __builtin_amdgcn_s_sleep(64);
    Work w;
    if (at < end) {
        w = work_of(locate(at));
        start(w);
    }
    while (at < end) {
        at += turn;
        Spot next{};
        if (at < end) next = locate(at);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = Sums{0.0f, 0.0f, 0.0f, 0.0f};
        if (w.blocks) {
            meet<0>();
            if (w.blocks == 1 && (w.depth & 127u)) {
                clear_tail<BM, kThreads, 1>(row_tile[0], w.depth);
                clear_tail<BN, kThreads, RUN>(col_tile[0], w.depth);
                meet<0>();
            }
            read_cols(0);
            meet<0>();
        }
        for (uint32_t b = 0; b < w.blocks; b += 2) {
            step(w, b, std::integral_constant<int, 0>{});
            if (b + 1 < w.blocks) step(w, b + 1, std::integral_constant<int, 1>{});
        }
        meet<0>();  // nobody reads LDS any more
        T *out = static_cast<T *>(a.out) + w.out;
        const uint32_t last_row = w.last_row, width = w.width;
        if (at < end) {
            w = work_of(next);
            start(w);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint32_t m = (wm * MT + i) * 16 + l;
#pragma unroll
            for (int j0 = 0; j0 < NT; j0 += RUN) {
                const uint32_t n = wn * NT * 16 + lane / 16 * (4 * RUN) + col_of(j0);
                if (m <= last_row && n < width) {
                    float v[RUN * 4];
#pragma unroll
                    for (int j = 0; j < RUN * 4; ++j) v[j] = acc[i][j0 + j / 4][j % 4];
                    store<T, RUN * 4>(out + (int64_t)m * a.out_stride + n, v, width - n,
                                      TURNED && a.accumulate);
                }
            }
        }
    }
    if constexpr (!TURNED) {  // the rows behind the last expert's
        const int64_t first = cut_offset(a.seg, a.seg.experts);
        for (int64_t r = first + blockIdx.x; r < a.seg.rows; r += gridDim.x) {
            T *row = static_cast<T *>(a.out) + r * a.out_stride;
            for (uint32_t n = threadIdx.x; n < a.width; n += kThreads) row[n] = (T)0.0f;
        }
    }
}

// The same for few rows an expert, where reading the weights is all there is: 16 * MT
// rows by 16 * NT columns, the blocks of 128 shared among the waves, each of which reads
// its operands into registers; what the waves have is added up in LDS.
template <class T, int MT, int NT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void thin_kernel(MulArgs a) {
    constexpr bool kExact = std::is_same<T, float>::value;
    constexpr int BM = MT * 16, BN = NT * 16, kStride = BN + 4, kAtOnce = 2;
    __shared__ __attribute__((aligned(16))) float part[WAVES][BM][kStride];
    const uint32_t lane = threadIdx.x % 64, l = lane % 16, g = lane / 16;
    const uint32_t wave = uniform(threadIdx.x / 64);
    Cursor cursor{0, 0};
    const Tile t = find_tile(a.seg, blockIdx.x, BM, a.col_tiles, cursor);
    if (t.expert >= a.seg.experts) {  // the rows behind the last expert's
        const int64_t first = cut_offset(a.seg, a.seg.experts);
        const uint32_t place = blockIdx.x - cursor.before * a.col_tiles;
        for (int64_t r = first + place; r < a.seg.rows; r += gridDim.x - cursor.before * a.col_tiles) {
            T *row = static_cast<T *>(a.out) + r * a.out_stride;
            for (uint32_t n = threadIdx.x; n < a.width; n += WAVES * 64) row[n] = (T)0.0f;
        }
        return;
    }
    const uint32_t expert = uniform(t.expert), n0 = uniform(t.column) * BN;
    const uint32_t row0 = uniform((uint32_t)t.begin);
    const uint32_t rows = uniform((uint32_t)t.end) - row0, last_row = (rows < BM ? rows : BM) - 1;
    const uint32_t last_col = (a.width - n0 < BN ? a.width - n0 : BN) - 1;
    const uint32_t blocks = (a.depth + 127) / 128;
    const uint8_t *row[MT], *col[NT];
    const float *row_scale[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const uint32_t m = i * 16 + l < last_row ? i * 16 + l : last_row;
        row[i] = a.rows + (int64_t)(row0 + m) * a.row_stride;
        row_scale[i] = a.row_scales + (int64_t)(row0 + m) * blocks;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const uint32_t n = j * 16 + l < last_col ? j * 16 + l : last_col;
        col[j] = a.cols + (int64_t)expert * a.col_matrix + (int64_t)(n0 + n) * a.col_stride;
    }
    const float *sw = a.col_scales + ((int64_t)expert * ((a.width + 127) / 128) + n0 / 128) * blocks;

    // The pieces g and g + 4 of a block; of the last, what is inside the row.
    const auto read = [&](const uint8_t *p, uint32_t b) {
        Quarter q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = b * 128 + (g + 4 * h) * 16;
            if (b * 128 + 128 <= a.depth) {
                q[h] = *reinterpret_cast<const Quarter *>(p + at);
            } else {
                q[h] = *reinterpret_cast<const Quarter *>(p + (at < a.depth ? at : 0u));
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int have = (int)a.depth - (int)(at + w * 4);
                    q[h][w] &= have >= 4 ? -1 : have <= 0 ? 0 : (int)((1u << (have * 8)) - 1u);
                }
            }
        }
        return __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7);
    };
    Sums acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Sums{0.0f, 0.0f, 0.0f, 0.0f};
    const auto go = [&](uint32_t b, auto count) {
        constexpr int N = decltype(count)::value;
        Frag r[N][MT], c[N][NT];
        float scale[N][MT];
#pragma unroll
        for (int u = 0; u < N; ++u) {
#pragma unroll
            for (int j = 0; j < NT; ++j) c[u][j] = read(col[j], b + u * WAVES);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                r[u][i] = read(row[i], b + u * WAVES);
                scale[u][i] = row_scale[i][b + u * WAVES];
            }
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const float cs = uniform_float(sw + b + u * WAVES);
            Operand<kExact> wide[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) wide[j] = operand<kExact>(c[u][j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const Operand<kExact> one = operand<kExact>(r[u][i]);
                const float s = scale[u][i] * cs;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const Sums p = multiply<kExact>(wide[j], one);
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[i][j][x] = fmaf(p[x], s, acc[i][j][x]);
                }
            }
        }
    };
    uint32_t b = wave;
    for (; b + WAVES * (kAtOnce - 1) < blocks; b += WAVES * kAtOnce)
        go(b, std::integral_constant<int, kAtOnce>{});
    for (; b < blocks; b += WAVES) go(b, std::integral_constant<int, 1>{});
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<Sums *>(&part[wave][i * 16 + l][j * 16 + g * 4]) = acc[i][j];
    __syncthreads();
    T *out = static_cast<T *>(a.out) + (int64_t)row0 * a.out_stride + n0;
    for (uint32_t u = threadIdx.x; u < BM * BN / 4; u += WAVES * 64) {
        const uint32_t m = u / (BN / 4), n = u % (BN / 4) * 4;
        if (m > last_row || n > last_col) continue;
        Sums s = *reinterpret_cast<const Sums *>(&part[0][m][n]);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += *reinterpret_cast<const Sums *>(&part[w][m][n]);
        const float v[4] = {s[0], s[1], s[2], s[3]};
        store<T, 4>(out + (int64_t)m * a.out_stride + n, v, last_col + 1 - n, false);
    }
}

bool good_sizes(int64_t rows, int64_t experts, int64_t width, int64_t depth) {
    const int64_t most = INT32_MAX - 1024;
    return rows >= 0 && rows < most && experts >= 1 && experts <= 65535 && width >= 1 &&
           width < most && depth >= 1 && depth < most;
}

// Rows of a tile are found by 32 bits from its first.
constexpr int64_t kMostStride = (1 << 24) - 1;

// Workgroups for so many tiles: those that the device holds at once, by their LDS, and a
// multiple of the XCDs.
unsigned groups_of(int64_t tiles, int bm, int bn) {
    const int64_t held = 256 * (bm + bn <= 192 ? 3 : bm + bn <= 256 ? 2 : 1);
    return (unsigned)(tiles < held ? (tiles + 7) / 8 * 8 : held);
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
    if (q.rows.stride > kMostStride || q.weights.stride > kMostStride) return SEGTOPK_NOT_SUPPORTED;
    return with_type(q.out.type, [&](auto v) -> int {
        using T = decltype(v);
        const auto go = [&](auto bm, auto bn, auto wm, auto wn) -> int {
            constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
            constexpr int WM = decltype(wm)::value, WN = decltype(wn)::value;
            a.col_tiles = (a.width + BN - 1) / BN;
            const int64_t tiles = tiles_most(q.num_rows, q.num_experts, BM);
            if (tiles > kMostBlocks / a.col_tiles) return SEGTOPK_NOT_SUPPORTED;
            a.seg.tiles_most = (uint32_t)tiles;
            return status(launch(product_kernel<T, BM, BN, WM, WN, false>,
                                 dim3(groups_of(tiles * a.col_tiles, BM, BN)), WM * WN * 64, stream,
                                 0, a));
        };
        using std::integral_constant;
        const auto thin = [&](auto mt, auto nt) -> int {
            constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value, kWaves = 4;
            a.col_tiles = (a.width + NT * 16 - 1) / (NT * 16);
            const int64_t tiles = tiles_most(q.num_rows, q.num_experts, MT * 16) + 1;
            if (tiles > kMostBlocks / a.col_tiles) return SEGTOPK_NOT_SUPPORTED;
            return status(launch(thin_kernel<T, MT, NT, kWaves>, dim3((unsigned)(tiles * a.col_tiles)),
                                 kWaves * 64, stream, 0, a));
        };
        const auto thin_by_width = [&](auto mt) -> int {
            const int64_t tiles = tiles_most(q.num_rows, q.num_experts, decltype(mt)::value * 16);
            return tiles * ((a.width + 63) / 64) >= 512   ? thin(mt, integral_constant<int, 4>{})
                   : tiles * ((a.width + 31) / 32) >= 512 ? thin(mt, integral_constant<int, 2>{})
                                                          : thin(mt, integral_constant<int, 1>{});
        };
        // By the rows of an average expert.  64 experts of 4096 to 2048, by 16, 32, 64 rows at a
        // time and by tiles of 128 x 128: 8 rows each 96, 111, 126, 124 us; 16 rows 104, 114,
        // 125, 122; 32 rows 192, 128, 135, 123.  Experts are not all alike, and one row too many
        // reads the weights again, hence 12 and 24.  Where tiles would leave most of the device
        // idle, the blocks shared among waves are quicker: one expert of 4096 to 8192, by 16, 32,
        // 64 rows, 16 rows 11, 15, 16 us; 64 rows 35, 23, 20; 256 rows 83, 57, 47.  By 64 rows
        // and by tiles of 64 x 128, with the squares below, in bf16 that one (192) 47 and 26; 2048
        // to 2048, 256 rows (48) 17 and 15; 1024 to 1024, 512 rows (40) 10 and 10, 8 experts to
        // 256, 128 rows each (32) 7 and 10.  In f32, whose products take twice as long, 192 squares
        // 56 and 36, 72 35 and 34, 64 17 and 20; 16 experts of 2048 to 768, 40 rows each (126) 17
        // and 19.  All of this is for depths of 1024 and more.  In shallower products the waves that
        // share an expert's blocks have few or none, and of many experts tiles of 64 x 128 would be
        // quicker: 64 to 2048, 16 rows each, weights in the last cache, by what is taken here and by
        // those, a depth of 128 14.5 and 7.4, 512 22 and 15, 1024 33 and 23; 128 to 1024, 8 rows
        // each, a depth of 128 11.4 and 7.6.  Under 200 squares all forms but those of 128 x 128 are
        // within a third of each other there.
        const int64_t each = (q.num_rows + q.num_experts - 1) / q.num_experts;
        const int64_t squares =
            tiles_most(q.num_rows, q.num_experts, 128) * ((a.width + 127) / 128);
        const bool few = squares < (each < 96 ? 200 : sizeof(T) == 2 ? 44 : 72);
        if (each <= (few ? 16 : 12)) return thin_by_width(integral_constant<int, 1>{});
        if (each <= (few ? 32 : 24)) return thin_by_width(integral_constant<int, 2>{});
        if (few) return thin_by_width(integral_constant<int, 4>{});
        // Larger tiles read less for each product, smaller ones fill the device and waste less
        // of an expert's last tile.  In bf16 by tiles of 64 x 128, 128 x 128 and 256 x 256: 64
        // experts of 4096 to 2048, 32 rows each 127, 130, 137 us; 128 rows 196, 188, 229; 256
        // rows 319, 263, 317; 128 experts, 512 rows each 1259, 941, 810.  In f32 1700, 1423 and
        // (256 x 128) 1406; 37 experts of 1008 to 777, 81 rows each 21, 30, 42.
        const integral_constant<int, 2> two;
        const integral_constant<int, 128> middle;
        if constexpr (sizeof(T) == 2) {
            const integral_constant<int, 256> large;
            const int64_t tiles =
                tiles_most(q.num_rows, q.num_experts, 256) * ((a.width + 255) / 256);
            if (each >= 384 && tiles >= 256) return go(large, large, two, integral_constant<int, 4>{});
        }
        if (squares < 512) return go(integral_constant<int, 64>{}, middle, two, two);
        return go(middle, middle, two, two);
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
    const auto tiles_of_size = [&](int64_t size) {
        return (a.width + size - 1) / size * ((a.height + size - 1) / size);
    };
    if (tiles_of_size(128) > kMostBlocks / q.num_experts || s.stride > kMostStride)
        return SEGTOPK_NOT_SUPPORTED;
    if (s.tiles) {
        const int r = queue_quantize_turned(q.dout, dout, q.rows, rows, seg, stream);
        if (r != SEGTOPK_OK) return r;
    }
    return with_type(d.type, [&](auto v) -> int {
        using T = decltype(v);
        using std::integral_constant;
        const auto go = [&](auto size, auto waves) -> int {
            constexpr int kSize = decltype(size)::value, kAcross = decltype(waves)::value;
            a.col_tiles = (a.width + kSize - 1) / kSize;
            a.row_tiles = (a.height + kSize - 1) / kSize;
            const int64_t tiles = (int64_t)a.col_tiles * a.row_tiles * q.num_experts;
            return status(launch(product_kernel<T, kSize, kSize, 2, kAcross, true>,
                                 dim3(groups_of(tiles, kSize, kSize)), kAcross * 128, stream, 0, a));
        };
        // As above, by tiles of 128 and 256, quantization included: 128 experts of 2048 x 4096,
        // 512 rows each 1743 and 1659 us, 128 rows 912 and 957; 16 of 2048 x 2048, 1024 rows 207
        // and 191, 128 rows 71 and 76; 8 of 4096 x 14336, 2048 rows 3278 and 2605; 60 of 336 x
        // 1410, 78 rows 46 and 55.
        if constexpr (sizeof(T) == 2)
            if (q.num_rows / q.num_experts >= 384 && tiles_of_size(256) * q.num_experts >= 512)
                return go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
        // Where tiles of 128 would leave most of the device idle, smaller ones: by 128 and 64, 1719
        // x 1123 (126 tiles), 2850 rows in f32, 55 and 44 us; 4 experts of 512 x 512 (64), 4096
        // rows in bf16, 24 and 18; 4096 x 1024 (256), 4096 rows, 54 and 55.
        if (tiles_of_size(128) * q.num_experts < 256)
            return go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
        return go(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    });
}
