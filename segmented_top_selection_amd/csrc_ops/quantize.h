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

// A tile: rows begin .. end of one expert's, of which it has the first `size` at most.
struct Tile {
    uint32_t expert;  // the number of experts: rows behind the last expert's; beyond it: none
    int64_t begin, end;
    uint32_t index, count;  // of the expert's tiles: this one, and the tiles of those before it
};

inline int64_t tiles_most(int64_t rows, int64_t experts, int64_t size) {
    return rows / size + (rows < experts ? rows : experts);
}

__device__ inline int64_t cut_offset(const Segments &s, uint32_t e) {
    const int64_t v = s.offsets[e];
    return v < 0 ? 0 : v > s.rows ? s.rows : v;
}

// Tile number `tile` when each expert's rows are cut into tiles of `size`, by a wave:
// 64 experts at a time, their tiles added up across the lanes.
__device__ inline Tile find_tile(const Segments &s, uint32_t tile, uint32_t size) {
    const uint32_t lane = __lane_id();
    uint32_t before = 0;
    for (uint32_t e0 = 0; e0 < s.experts; e0 += 64) {
        const uint32_t e = e0 + lane;
        int64_t begin = 0, end = 0;
        if (e < s.experts) {
            begin = cut_offset(s, e);
            end = cut_offset(s, e + 1);
        }
        const uint32_t n = end > begin ? (uint32_t)((end - begin + size - 1) / size) : 0u;
        uint32_t sum = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t v = __shfl_up(sum, d);
            if ((int)lane >= d) sum += v;
        }
        const uint32_t all = __shfl(sum, 63);
        if (tile - before < all) {
            const uint64_t at = __ballot(before + sum > tile);
            const int l = __builtin_ctzll(at);
            Tile t;
            t.expert = e0 + l;
            t.count = before + __shfl(sum, l) - __shfl(n, l);
            t.index = tile - t.count;
            const int64_t b = __shfl(begin, l);
            t.begin = b + (int64_t)t.index * size;
            t.end = __shfl(end, l);
            return t;
        }
        before += all;
    }
    return {s.experts, 0, 0, 0, before};
}

// Rows transposed: element (c, r) at q[c * stride + r], r counted over the tiles of 128
// rows, zeros behind an expert's last; scales[tile * width + c].
struct Turned {
    uint8_t *q;
    float *scales;
    int64_t stride;
    uint32_t width;
};

int queue_quantize_turned(const segtopk_rows &x, const Turned &t, const Segments &seg,
                          hipStream_t stream);

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
