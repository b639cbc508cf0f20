// sort_ids.hip -- the stable sort of small integers (expert or token ids):
// order = stable argsort of key_i, where key_i = id_i inside [0, S) and S
// otherwise; position = its inverse; offsets[s] = #{i : key_i < s}.
//
// Least-significant-digit radix passes of at most 9 bits.  A pass splits the
// items into consecutive chunks, one workgroup of 16 waves each, and a chunk
// into 16 consecutive parts, one for each wave:
//   count_kernel    digit histogram of each chunk
//   scatter_kernel  where a chunk's items of digit d start: all items of smaller
//                   digits, and those of d in earlier chunks and waves; then
//                   each wave takes its items 64 at a time, ranks equal digits
//                   by the lanes below (one ballot a bit) and writes them.
// One chunk needs no count_kernel.  Up to 511 segments take one pass.  No atomic
// decides an order, so results are the same every time.
//
// Bound by launches and by the latency of the dependent steps, not by its
// bytes (16 to 20 an item).
#include "ops_common.h"

namespace segtopk_ops {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBits = 9;  // the waves' counters then take 37 KB of LDS
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int64_t kOneChunk = 4096;   // items that one workgroup sorts alone
constexpr int64_t kMinChunk = 2048;
constexpr int64_t kMaxChunks = 128;

struct SortArgs {
    const void *ids;       // first pass: the caller's ids
    const uint32_t *key_in;  // later passes: keys and the slots they came from
    const uint32_t *slot_in;
    uint32_t *key_out;     // nullptr: not wanted
    uint32_t *slot_out;
    int32_t *position;     // last pass, or nullptr
    int64_t *offsets;      // of a sort in one pass, or nullptr
    uint32_t *hist;        // [chunks][bins]
    uint32_t n, segments, chunk, chunks, shift, bins, bits;
    uint32_t wide;         // ids of 64 bits
};

template <bool FIRST> __device__ inline uint32_t sort_key(const SortArgs &a, uint32_t i) {
    if (!FIRST) return a.key_in[i];
    const int64_t id = a.wide ? static_cast<const int64_t *>(a.ids)[i]
                              : (int64_t) static_cast<const int32_t *>(a.ids)[i];
    return (id >= 0 && id < (int64_t)a.segments) ? (uint32_t)id : a.segments;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void count_kernel(SortArgs a) {
    __shared__ uint32_t cnt[kMaxBins];
    const uint32_t t = threadIdx.x;
    if (t < a.bins) cnt[t] = 0u;
    __syncthreads();
    const uint32_t b = blockIdx.x * a.chunk;
    const uint32_t e = min(a.n, b + a.chunk);
    for (uint32_t i = b + t; i < e; i += kSortThreads)
        atomicAdd(&cnt[(sort_key<FIRST>(a, i) >> a.shift) & ((1u << a.bits) - 1u)], 1u);
    __syncthreads();
    if (t < a.bins) a.hist[(size_t)blockIdx.x * a.bins + t] = cnt[t];
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void scatter_kernel(SortArgs a) {
    extern __shared__ uint32_t lds[];
    uint32_t *const whist = lds;                       // [waves][bins]
    uint32_t *const wave_total = lds + kSortWaves * a.bins;  // [waves]
    uint32_t *const total = wave_total + kSortWaves;   // [bins]
    uint32_t *const before = total + a.bins;           // [bins]
    const uint32_t t = threadIdx.x, lane = t & 63u, w = t >> 6;
    const uint32_t mask = (1u << a.bits) - 1u;
    const uint32_t b = blockIdx.x * a.chunk;
    const uint32_t e = min(a.n, b + a.chunk);
    const uint32_t part = a.chunk / kSortWaves;  // a multiple of 64
    const uint32_t wb = min(e, b + w * part), we = min(e, wb + part);

    for (uint32_t i = t; i < kSortWaves * a.bins; i += kSortThreads) whist[i] = 0u;
    if (t < a.bins) total[t] = before[t] = 0u;
    __syncthreads();
    for (uint32_t i = wb + lane; i < we; i += 64u)
        atomicAdd(&whist[w * a.bins + ((sort_key<FIRST>(a, i) >> a.shift) & mask)], 1u);
    // Rows of the histograms of all chunks, shared out among groups of threads.
    if (a.chunks > 1) {
        uint32_t width = 64;
        while (width < a.bins) width <<= 1;
        const uint32_t d = t & (width - 1u), groups = kSortThreads / width;
        if (d < a.bins) {
            uint32_t all = 0, mine = 0;
#pragma unroll 8
            for (uint32_t c = t / width; c < a.chunks; c += groups) {
                const uint32_t v = a.hist[(size_t)c * a.bins + d];
                all += v;
                mine += c < blockIdx.x ? v : 0u;
            }
            atomicAdd(&total[d], all);  // integers: any order gives the same sum
            atomicAdd(&before[d], mine);
        }
    }
    __syncthreads();
    // Exclusive prefix of the totals over the digits, one thread a digit.
    uint32_t own = 0;
    if (t < a.bins) {
        if (a.chunks > 1) own = total[t];
        else
            for (int i = 0; i < kSortWaves; ++i) own += whist[i * a.bins + t];
    }
    uint32_t run = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(run, d);
        if (lane >= (uint32_t)d) run += v;
    }
    if (lane == 63u) wave_total[w] = run;
    __syncthreads();
    if (t < a.bins) {
        uint32_t base = run - own;
        for (uint32_t i = 0; i < w; ++i) base += wave_total[i];
        if (a.offsets && blockIdx.x == 0) a.offsets[t] = base;  // bins = segments + 1 then
        base += before[t];
        for (int i = 0; i < kSortWaves; ++i) {
            const uint32_t c = whist[i * a.bins + t];
            whist[i * a.bins + t] = base;
            base += c;
        }
    }
    __syncthreads();
    // A wave's items in order, 64 at a time; its counters are its own.
    volatile uint32_t *const next = whist + w * a.bins;
    for (uint32_t i0 = wb; i0 < we; i0 += 64u) {
        const uint32_t i = i0 + lane;
        const bool live = i < we;
        const uint32_t key = live ? sort_key<FIRST>(a, i) : 0u;
        const uint32_t digit = (key >> a.shift) & mask;
        uint64_t peers = __ballot(live);
        for (uint32_t j = 0; j < a.bits; ++j) {
            const uint64_t ones = __ballot((digit >> j) & 1u);
            peers &= ((digit >> j) & 1u) ? ones : ~ones;
        }
        const uint32_t rank = __popcll(peers & ((1ull << lane) - 1ull));
        uint32_t at = 0;
        if (live) at = next[digit];
        __builtin_amdgcn_wave_barrier();
        if (live && rank == 0) next[digit] = at + (uint32_t)__popcll(peers);
        __builtin_amdgcn_wave_barrier();
        if (live) {
            const uint32_t slot = FIRST ? i : a.slot_in[i];
            at += rank;
            if (a.key_out) a.key_out[at] = key;
            if (a.slot_out) a.slot_out[at] = slot;
            if (a.position) a.position[slot] = (int32_t)at;
        }
    }
}

// offsets[s] of a sort in several passes: the first place of a key >= s.
__global__ void offsets_kernel(const uint32_t *sorted, uint32_t n, uint32_t segments,
                               int64_t *offsets) {
    const uint32_t s = blockIdx.x * blockDim.x + threadIdx.x;
    if (s > segments) return;
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + ((hi - lo) >> 1);
        if (sorted[mid] < s) lo = mid + 1;
        else hi = mid;
    }
    offsets[s] = lo;
}

struct SortPlan {
    int passes, bits;
    uint32_t bins, chunk, chunks;
    size_t hist_bytes, pair_bytes, bytes;
};

SortPlan sort_plan(int64_t n, int64_t segments) {
    SortPlan p{};
    if (segments + 1 <= kMaxBins) {
        p.passes = 1;
        p.bins = (uint32_t)(segments + 1);
        p.bits = 1;
        while ((1u << p.bits) < p.bins) ++p.bits;
    } else {
        int bits = 1;
        while (((int64_t)1 << bits) < segments + 1) ++bits;
        p.passes = (bits + kMaxBits - 1) / kMaxBits;
        p.bits = (bits + p.passes - 1) / p.passes;
        p.bins = 1u << p.bits;
    }
    int64_t chunk = n;
    if (n > kOneChunk) {
        chunk = (n + kMaxChunks - 1) / kMaxChunks;
        if (chunk < kMinChunk) chunk = kMinChunk;
    }
    chunk = (chunk + kSortThreads - 1) / kSortThreads * kSortThreads;
    if (chunk < kSortThreads) chunk = kSortThreads;
    p.chunk = (uint32_t)chunk;
    p.chunks = n ? (uint32_t)((n + chunk - 1) / chunk) : 1u;
    p.hist_bytes = p.chunks > 1 ? ((size_t)p.chunks * p.bins * 4 + 255) & ~(size_t)255 : 0;
    // Keys and slots between the passes, in two buffers taken in turn from
    // three passes on, and the keys in order where offsets are searched in them.
    p.pair_bytes = ((size_t)n * 4 + 255) & ~(size_t)255;
    p.bytes = p.hist_bytes + (p.passes > 1 ? 5 : 0) * p.pair_bytes;
    return p;
}

}  // namespace

size_t sort_workspace(int64_t n, int64_t segments) { return sort_plan(n, segments).bytes; }

hipError_t queue_sort(const void *ids, int id_type, int64_t n, int64_t segments, int32_t *order,
                      int32_t *position, int64_t *offsets, uint32_t *sorted, void *workspace,
                      hipStream_t stream) {
    const SortPlan p = sort_plan(n, segments);
    char *ws = static_cast<char *>(workspace);
    uint32_t *pair[2][2];
    for (int i = 0; i < 4; ++i)
        pair[i >> 1][i & 1] = reinterpret_cast<uint32_t *>(ws + p.hist_bytes + i * p.pair_bytes);
    if (p.passes > 1 && !sorted)
        sorted = reinterpret_cast<uint32_t *>(ws + p.hist_bytes + 4 * p.pair_bytes);
    SortArgs a{};
    a.ids = ids;
    a.hist = reinterpret_cast<uint32_t *>(ws);
    a.n = (uint32_t)n;
    a.segments = (uint32_t)segments;
    a.chunk = p.chunk;
    a.chunks = p.chunks;
    a.bins = p.bins;
    a.bits = (uint32_t)p.bits;
    a.wide = id_type == SEGTOPK_KEY_I64;
    const size_t lds = 4 * ((size_t)(kSortWaves + 2) * p.bins + kSortWaves);
    hipError_t err;
    for (int i = 0; i < p.passes; ++i) {
        const bool last = i == p.passes - 1;
        a.shift = (uint32_t)(i * p.bits);
        a.key_in = i ? pair[(i - 1) & 1][0] : nullptr;
        a.slot_in = i ? pair[(i - 1) & 1][1] : nullptr;
        a.key_out = last ? sorted : pair[i & 1][0];
        a.slot_out = last ? reinterpret_cast<uint32_t *>(order) : pair[i & 1][1];
        a.position = last ? position : nullptr;
        a.offsets = p.passes == 1 ? offsets : nullptr;
        if (p.chunks > 1) {
            hipLaunchKernelGGL(i ? count_kernel<false> : count_kernel<true>, dim3(p.chunks),
                               dim3(kSortThreads), 0, stream, a);
            if ((err = hipGetLastError()) != hipSuccess) return err;
        }
        hipLaunchKernelGGL(i ? scatter_kernel<false> : scatter_kernel<true>, dim3(p.chunks),
                           dim3(kSortThreads), lds, stream, a);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    if (p.passes > 1 && offsets) {
        hipLaunchKernelGGL(offsets_kernel, dim3((unsigned)((segments + 256) / 256)), dim3(256), 0,
                           stream, sorted, (uint32_t)n, (uint32_t)segments, offsets);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace segtopk_ops

using namespace segtopk_ops;

extern "C" int64_t segtopk_sort_ids_workspace(int64_t n, int64_t num_segments) {
    if (n < 0 || n > INT32_MAX || num_segments < 0 || num_segments >= INT32_MAX) return 0;
    return (int64_t)sort_workspace(n, num_segments);
}

extern "C" int segtopk_sort_ids(const void *ids, int32_t id_type, int64_t n, int64_t num_segments,
                                int32_t *order, int32_t *position, int64_t *offsets,
                                void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    const int ib = index_bytes(id_type);
    if (!ib || n < 0 || n > INT32_MAX || num_segments < 0 || num_segments >= INT32_MAX)
        return SEGTOPK_INVALID_ARGUMENT;
    if (!offsets || !aligned(offsets, 8)) return SEGTOPK_INVALID_ARGUMENT;
    if (n && (!ids || !aligned(ids, ib) || !order || !aligned(order, 4) || !position ||
              !aligned(position, 4)))
        return SEGTOPK_INVALID_ARGUMENT;
    const size_t need = sort_workspace(n, num_segments);
    if (need && (!workspace || !aligned(workspace, 256))) return SEGTOPK_INVALID_ARGUMENT;
    if (workspace_bytes < 0 || (size_t)workspace_bytes < need) return SEGTOPK_SCRATCH_TOO_SMALL;
    return status(queue_sort(ids, id_type, n, num_segments, order, position, offsets, nullptr,
                             workspace, stream));
}
