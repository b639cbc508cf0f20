// ops_common.h -- what the operators around the selection share: element
// types, 16-byte pieces of rows that may start at any element, wave
// reductions, and the host's checks and launch arithmetic.
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "segtopk.h"

namespace segtopk_ops {

constexpr int kOpThreads = 256;

// One 16-byte piece of a row.  Rows may start at any element (odd widths,
// slices of wider rows), so the type claims the element's alignment only;
// gfx950 serves such pieces with the same 16-byte memory instructions.
template <class T> struct Piece {
    static constexpr int N = 16 / (int)sizeof(T);
    typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
    typedef T mem __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
    typedef float f32 __attribute__((ext_vector_type(16 / sizeof(T))));
};

// STREAM: past the caches, for what is not touched again soon.
template <bool STREAM = false, class T>
__device__ inline typename Piece<T>::vec load_piece(const T *p) {
    const auto *q = reinterpret_cast<const typename Piece<T>::mem *>(p);
    return STREAM ? __builtin_nontemporal_load(q) : *q;
}
template <bool STREAM = false, class T>
__device__ inline void store_piece(T *p, typename Piece<T>::vec v) {
    auto *q = reinterpret_cast<typename Piece<T>::mem *>(p);
    if (STREAM) __builtin_nontemporal_store((typename Piece<T>::mem)v, q);
    else *q = v;
}
template <class T>
__device__ inline typename Piece<T>::f32 widen(typename Piece<T>::vec v) {
    return __builtin_convertvector(v, typename Piece<T>::f32);
}
// Rounds to nearest even.
template <class T>
__device__ inline typename Piece<T>::vec narrow(typename Piece<T>::f32 v) {
    return __builtin_convertvector(v, typename Piece<T>::vec);
}

__device__ inline float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Lane i's value from the lane that step D of a butterfly pairs it with; the
// steps below 16 pair lanes whose halves already agree, so that a mirror serves.
template <int D> __device__ inline uint32_t partner(uint32_t v) {
    if constexpr (D == 1) return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, false);
    else if constexpr (D == 2) return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, false);
    else if constexpr (D == 4) return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xF, 0xF, false);
    else if constexpr (D == 8) return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xF, 0xF, false);
    else return __shfl_xor(v, D);
}
template <int D> __device__ inline float partner(float v) {
    return __uint_as_float(partner<D>(__float_as_uint(v)));
}
template <int D> __device__ inline double partner(double v) {
    const uint32_t lo = partner<D>((uint32_t)__double2loint(v));
    const uint32_t hi = partner<D>((uint32_t)__double2hiint(v));
    return __hiloint2double((int)hi, (int)lo);
}

// f over the L lanes (16 or 64) of a lane's own, for all of them.
template <int L, class X, class F> __device__ inline X join(X v, F f) {
    v = f(v, partner<1>(v));
    v = f(v, partner<2>(v));
    v = f(v, partner<4>(v));
    v = f(v, partner<8>(v));
    if constexpr (L > 16) {
        v = f(v, partner<16>(v));
        v = f(v, partner<32>(v));
    }
    return v;
}
// ---- host ---------------------------------------------------------------
// Workgroups of kOpThreads that one launch holds: fewer than 2^32 threads.
constexpr int64_t kMostBlocks = (1 << 24) - 1;
inline int element_bytes(int type) {
    return type == SEGTOPK_KEY_F32 ? 4
           : (type == SEGTOPK_KEY_BF16 || type == SEGTOPK_KEY_F16) ? 2 : 0;
}
inline int index_bytes(int type) {
    return type == SEGTOPK_KEY_I32 ? 4 : type == SEGTOPK_KEY_I64 ? 8 : 0;
}
inline bool aligned(const void *p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes) == 0;
}
// A matrix of at least one row that the call reads or writes.
inline bool good_rows(const segtopk_rows *m, int64_t width) {
    const int b = m ? element_bytes(m->type) : 0;
    return b && m->data && aligned(m->data, b) && m->stride >= width;
}
// Whether an output of so many bytes is stored past the caches: with the inputs it
// no longer fits the 256 MB that the last of them holds.
inline bool streams(int64_t bytes) { return bytes >= ((int64_t)128 << 20); }
inline int status(hipError_t e) { return e == hipSuccess ? SEGTOPK_OK : SEGTOPK_HIP_ERROR; }

// Queues a kernel, and says itself whether that failed: the runtime's last error may
// be another call's.  (It is also a little quicker than the <<<>>> form, 2.2 us
// against 2.4.)
template <class T> struct Given { using type = T; };
template <class... P>
inline hipError_t launch(void (*kernel)(P...), dim3 grid, unsigned threads, hipStream_t stream,
                         size_t lds, typename Given<P>::type... args) {
    void *given[] = {const_cast<void *>(static_cast<const void *>(&args))...};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, dim3(threads), given, lds,
                           stream);
}

// Calls f with a value of the element type.
template <class F> inline int with_type(int type, F f) {
    switch (type) {
    case SEGTOPK_KEY_F32: return f(float{});
    case SEGTOPK_KEY_BF16: return f(__bf16{});
    default: return f(_Float16{});
    }
}

// Memory to clear beside other work, from a multiple of 16 bytes on, an even
// number of them.  A thread stores 16 bytes once where the grid allows it: a
// device full of such workgroups writes in the order of addresses, 1 GiB at
// 6.3 TB/s by workgroups of 1024 threads, the size of the sort's beside which they
// run (6.9 by 256), where 64 KiB to a workgroup reach 4.9.
struct Fill {
    void *data;
    uint64_t bytes;
    uint32_t stream;
};
constexpr int64_t kFillBlocks = 1 << 20;  // of a launch, at most
inline uint32_t fill_blocks(const Fill &f, uint32_t threads) {
    const uint64_t n = (f.bytes + (uint64_t)threads * 16 - 1) / ((uint64_t)threads * 16);
    return (uint32_t)(n < (uint64_t)kFillBlocks ? n : (uint64_t)kFillBlocks);
}

// What the workgroup `block` of the `blocks` that clear does.
__device__ inline void clear(const Fill &f, uint32_t block, uint32_t blocks) {
    float *const data = static_cast<float *>(f.data);
    const uint64_t pieces = f.bytes / 16;
    for (uint64_t i = (uint64_t)block * blockDim.x + threadIdx.x; i < pieces;
         i += (uint64_t)blocks * blockDim.x) {
        if (f.stream) store_piece<true>(data + i * 4, Piece<float>::vec(0.0f));
        else store_piece(data + i * 4, Piece<float>::vec(0.0f));
    }
    const uint32_t rest = (uint32_t)(f.bytes % 16) / 2;
    if (block == 0 && threadIdx.x < rest)
        reinterpret_cast<uint16_t *>(data + pieces * 4)[threadIdx.x] = 0;
}

// The stable sort of n ids (sort_ids.hip), for the operators that need it
// inside: any of `order`, `position`, `offsets` and `sorted` (the ids in order,
// num_segments for a dropped one) may be nullptr.  `fill`, if given, is cleared
// beside it: the sort leaves most of the device idle.
size_t sort_workspace(int64_t n, int64_t num_segments);
hipError_t queue_sort(const void *ids, int id_type, int64_t n, int64_t num_segments, int32_t *order,
                      int32_t *position, int64_t *offsets, uint32_t *sorted, void *workspace,
                      hipStream_t stream, const Fill *fill = nullptr);

}  // namespace segtopk_ops
