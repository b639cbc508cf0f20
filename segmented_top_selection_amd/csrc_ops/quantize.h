// quantize.h -- what the 8-bit operators share: the rows of a batch as the experts'
// segments cut them into tiles, and rows transposed in 8 bits.
#pragma once

#include "ops_common.h"

namespace segtopk_ops {

// The experts' rows: offsets as sort_ids gives them, in device memory.
struct Segments {
    const int64_t *offsets;
    int64_t rows;
    uint32_t experts;
    uint32_t tiles_most;  // no batch of so many rows and experts has more tiles
};

inline int64_t tiles_most(int64_t rows, int64_t experts, int64_t size) {
    return rows / size + (rows < experts ? rows : experts);
}

__device__ inline int64_t cut_offset(const Segments &s, uint32_t e) {
    const int64_t v = s.offsets[e];
    return v < 0 ? 0 : v > s.rows ? s.rows : v;
}

// 64 experts' rows, one to a lane, and their tiles of `size` rows with those before them.
struct Strip {
    int64_t begin, end;
    uint32_t own, upto;  // the expert's tiles; all of the strip up to it, its own too
};
__device__ inline Strip strip_of(const Segments &s, uint32_t first, uint32_t size) {
    const uint32_t lane = __lane_id(), e = first + lane;
    Strip r{0, 0, 0, 0};
    if (e < s.experts) {
        r.begin = cut_offset(s, e);
        r.end = cut_offset(s, e + 1);
    }
    r.own = r.end > r.begin ? (uint32_t)((r.end - r.begin + size - 1) / size) : 0u;
    r.upto = r.own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(r.upto, d);
        if ((int)lane >= d) r.upto += v;
    }
    return r;
}

// The tiles of all experts, by a wave.
__device__ inline uint32_t count_tiles(const Segments &s, uint32_t size) {
    uint32_t sum = 0;
    for (uint32_t e = __lane_id(); e < s.experts; e += 64) {
        const int64_t begin = cut_offset(s, e), end = cut_offset(s, e + 1);
        sum += end > begin ? (uint32_t)((end - begin + size - 1) / size) : 0u;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    return sum;
}

// Where a search for tiles has come to: tiles are asked for in rising order.
struct Cursor {
    uint32_t first, before;  // the strip's first expert, and the tiles before it
};

// A tile: rows begin .. end of one expert's, of which it has the first `size` at most.
struct Tile {
    uint32_t expert;  // the number of experts: there is no such tile
    uint32_t column;
    int64_t begin, end;
};

// Tiles down first within groups of so many, so that neighbours share rows and columns.
constexpr uint32_t kGroupTiles = 8;
struct Place {
    uint32_t down, across;
};
__device__ inline Place place_of(uint32_t at, uint32_t high, uint32_t across) {
    const uint32_t group = at / (kGroupTiles * across) * kGroupTiles;
    at -= group * across;
    const uint32_t rest = high - group < kGroupTiles ? high - group : kGroupTiles;
    return {group + at % rest, at / rest};
}

// Tile number `tile`, `across` of them to each `size` rows, when each expert's rows are
// cut so; by a wave.
__device__ inline Tile find_tile(const Segments &s, uint32_t tile, uint32_t size, uint32_t across,
                                 Cursor &c) {
    for (; c.first < s.experts; c.first += 64) {
        const Strip r = strip_of(s, c.first, size);
        const uint32_t all = __shfl(r.upto, 63);
        if (tile - c.before * across < all * across) {
            const int l = __builtin_ctzll(__ballot((c.before + r.upto) * across > tile));
            const uint32_t own = __shfl(r.own, l), first = c.before + __shfl(r.upto, l) - own;
            const Place at = place_of(tile - first * across, own, across);
            return {c.first + l, at.across, __shfl(r.begin, l) + (int64_t)at.down * size,
                    __shfl(r.end, l)};
        }
        c.before += all;
    }
    return {s.experts, 0, 0, 0};
}

// The tiles before expert e's, and its own; by a wave.
struct Range {
    uint32_t first, count;
};
__device__ inline Range tiles_of(const Segments &s, uint32_t e, uint32_t size, Cursor &c) {
    for (;;) {
        const Strip r = strip_of(s, c.first, size);
        if (e - c.first < 64) {
            const int l = (int)(e - c.first);
            const uint32_t own = __shfl(r.own, l);
            return {c.before + __shfl(r.upto, l) - own, own};
        }
        c.before += __shfl(r.upto, 63);
        c.first += 64;
    }
}

// Rows transposed: element (c, r) at q[c * stride + r], r counted over the tiles of 128
// rows, zeros behind an expert's last; scales[tile * width + c].
struct Turned {
    uint8_t *q;
    float *scales;
    int64_t stride;
    uint32_t width;
};

// Both in one launch: of few rows each alone is as slow (60 experts of 336 and 1410 columns,
// 4662 rows in fp16: 9.6 and 12.1 us).
int queue_quantize_turned(const segtopk_rows &one, const Turned &one_turned, const segtopk_rows &two,
                          const Turned &two_turned, const Segments &seg, hipStream_t stream);

// Rows in 8 bits.
inline bool good_rows8(const segtopk_rows *m, int64_t width) {
    return m && m->type == SEGTOPK_E4M3 && m->data && aligned(m->data, 16) && m->stride >= width &&
           m->stride % 16 == 0;
}
inline bool good_matrices8(const segtopk_matrices *m, int64_t width) {
    return m && m->type == SEGTOPK_E4M3 && m->data && aligned(m->data, 16) && m->stride >= width &&
           m->stride % 16 == 0 && m->matrix_stride >= 0 && m->matrix_stride % 16 == 0;
}

}  // namespace segtopk_ops
