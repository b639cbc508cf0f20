// sort_ids.hip -- the stable sort of small integers (expert or token ids):
// order = stable argsort of key_i, where key_i = id_i inside [0, S) and S
// otherwise; position = its inverse; offsets[s] = #{i : key_i < s}.
//
// Few ids:
//   rank_kernel     counts for each item those before it, n^2 comparisons spread
//                   over the device
// Somewhat more, among many segments:
//   rank_kernel     sorts chunks of 1024 that way,
//   merge_kernel    and this counts for each item those before it in the others
// More: least-significant-digit radix passes of at most 9 bits, by workgroups of
// 16 waves.  A block of up to 8192 items stays in registers, eight to a lane, each
// wave holding consecutive items.  A wave takes its items 64 at a time and ranks
// equal digits by the lanes below (one ballot a bit) and the wave's own counters in
// LDS; the counters of the 16 waves, summed digit by digit, then say where each
// wave's items of a digit start.
//   count_kernel    the digit histogram of each chunk,
//   scatter_kernel  and the pass itself, every workgroup adding up the histograms
//                   of the chunks before its own
// Up to 511 segments take one pass, up to 262143 two.  No atomic decides an order,
// so results are the same every time.
//
// Bound by launches and by the latency of the dependent steps, not by its
// bytes (16 to 20 an item): 512 ids among 64 segments take 2.7 us, 8000 among 128
// 8.8, 65536 among 128 8.8, 32768 among 131072 25.7, a million among 256 26.
#include "ops_common.h"

namespace segtopk_ops {
namespace {

constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / 64;
constexpr int kItems = 8;  // of a lane
constexpr uint32_t kBlock = kSortThreads * kItems;
constexpr int kMaxBits = 9;
constexpr uint32_t kMaxBins = 1u << kMaxBits;
constexpr int64_t kMinChunk = 1024;

struct SortArgs {
    const void *ids;       // first pass: the caller's ids
    const uint32_t *key_in;  // later passes: keys and the slots they came from
    const uint32_t *slot_in;
    uint32_t *key_out;     // nullptr: not wanted
    uint32_t *slot_out;
    int32_t *position;     // last pass, or nullptr
    int64_t *offsets;      // or nullptr: searched in the sorted keys afterwards
    uint32_t *hist;        // [chunks][bins]
    uint32_t n, segments, chunk, chunks, shift, bins, bits;
    uint32_t wide;         // ids of 64 bits
    Fill fill;             // cleared by the workgroups past `chunks`
};

template <bool FIRST> __device__ inline uint32_t sort_key(const SortArgs &a, uint32_t i) {
    if (!FIRST) return a.key_in[i];
    const int64_t id = a.wide ? static_cast<const int64_t *>(a.ids)[i]
                              : (int64_t) static_cast<const int32_t *>(a.ids)[i];
    return (id >= 0 && id < (int64_t)a.segments) ? (uint32_t)id : a.segments;
}

// The items of one block in registers: lane l of wave w holds items
// w * 64 * items + r * 64 + l, r below `items`.
struct Items {
    uint32_t key[kItems], rank[kItems];
    uint32_t first, items, count;  // of the block; item r is live below count
    __device__ uint32_t at(int r) const { return first + (uint32_t)r * 64u; }
    __device__ bool live(int r) const { return (uint32_t)r < items && at(r) < count; }
};

// Counts the wave's items by digit in `mine` (zero before), and ranks each among
// those before it in the wave.
__device__ inline void rank_items(Items &x, uint32_t shift, uint32_t bits, uint32_t *mine) {
    const uint32_t mask = (1u << bits) - 1u;
    uint32_t below[kItems], peers[kItems];  // lanes of the same digit: those below, all
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        if ((uint32_t)r >= x.items) break;
        const uint32_t digit = (x.key[r] >> shift) & mask;
        const uint64_t live = __ballot(x.live(r));
        uint32_t lo = (uint32_t)live, hi = (uint32_t)(live >> 32);
#pragma unroll
        for (int j = 0; j < kMaxBits; ++j) {  // bits past the digit's are all zero
            const uint32_t bit = 0u - ((digit >> j) & 1u);
            const uint64_t ones = __ballot(bit != 0u);
            lo &= ~((uint32_t)ones ^ bit);
            hi &= ~((uint32_t)(ones >> 32) ^ bit);
        }
        below[r] = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0u));
        peers[r] = (uint32_t)(__popc(lo) + __popc(hi));
    }
    volatile uint32_t *const next = mine;
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        if ((uint32_t)r >= x.items) break;
        const uint32_t digit = (x.key[r] >> shift) & mask;
        uint32_t before = 0;
        if (x.live(r)) before = next[digit];
        __builtin_amdgcn_wave_barrier();
        if (x.live(r) && below[r] == 0) next[digit] = before + peers[r];
        __builtin_amdgcn_wave_barrier();
        x.rank[r] = before + below[r];
    }
}

// Exclusive prefix over the digits, thread d holding digit d's count.
__device__ inline uint32_t digit_prefix(uint32_t own, uint32_t *wave_total) {
    const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
    uint32_t run = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(run, d);
        if (lane >= (uint32_t)d) run += v;
    }
    if (lane == 63u) wave_total[w] = run;
    __syncthreads();
    uint32_t base = run - own;
    for (uint32_t i = 0; i < w; ++i) base += wave_total[i];
    return base;
}

// Turns the waves' counts of digit d into the places where their items start,
// from `base` on; returns where the next block's start.
__device__ inline uint32_t wave_starts(uint32_t *whist, uint32_t bins, uint32_t d, uint32_t base) {
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; ++w) {
        const uint32_t c = whist[w * bins + d];
        whist[w * bins + d] = base;
        base += c;
    }
    return base;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void count_kernel(SortArgs a) {
    __shared__ uint32_t cnt[kMaxBins];
    if (blockIdx.x >= a.chunks) return clear(a.fill, blockIdx.x - a.chunks, gridDim.x - a.chunks);
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
    __shared__ uint32_t whist[kSortWaves * kMaxBins], wave_total[kSortWaves];
    __shared__ uint32_t total[kMaxBins], before[kMaxBins];
    if (blockIdx.x >= a.chunks) return clear(a.fill, blockIdx.x - a.chunks, gridDim.x - a.chunks);
    const uint32_t t = threadIdx.x, lane = t & 63u, w = t >> 6;
    const uint32_t b = blockIdx.x * a.chunk, e = min(a.n, b + a.chunk);
    const uint32_t block = min(a.chunk, kBlock);
    Items x;
    x.items = block / kSortThreads;
    const uint32_t in_block = w * 64u * x.items + lane;
    x.first = b + in_block;
    x.count = e;
#pragma unroll
    for (int r = 0; r < kItems; ++r) x.key[r] = x.live(r) ? sort_key<FIRST>(a, x.at(r)) : 0u;
    if (t < a.bins) total[t] = before[t] = 0u;
    for (uint32_t i = t; i < kSortWaves * a.bins; i += kSortThreads) whist[i] = 0u;
    __syncthreads();
    {   // Rows of the histograms of all chunks, shared out among groups of threads.
        uint32_t width = 64;
        while (width < a.bins) width <<= 1;
        const uint32_t d = t & (width - 1u), groups = kSortThreads / width;
        if (d < a.bins) {
            uint32_t all = 0, mine = 0;
            for (uint32_t c0 = t / width; c0 < a.chunks; c0 += 8u * groups) {
                uint32_t v[8];
#pragma unroll
                for (uint32_t j = 0; j < 8u; ++j) {
                    const uint32_t c = c0 + j * groups;
                    v[j] = c < a.chunks ? a.hist[(size_t)c * a.bins + d] : 0u;
                }
#pragma unroll
                for (uint32_t j = 0; j < 8u; ++j) {
                    all += v[j];
                    mine += c0 + j * groups < blockIdx.x ? v[j] : 0u;
                }
            }
            atomicAdd(&total[d], all);  // integers: any order gives the same sum
            atomicAdd(&before[d], mine);
        }
    }
    rank_items(x, a.shift, a.bits, whist + w * a.bins);
    __syncthreads();
    uint32_t base = digit_prefix(t < a.bins ? total[t] : 0u, wave_total);
    if (t < a.bins) {
        if (a.offsets && blockIdx.x == 0) a.offsets[t] = base;  // one pass: bins = segments + 1
        base += before[t];
    }
    for (uint32_t b0 = b;;) {
        if (t < a.bins) base = wave_starts(whist, a.bins, t, base);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kItems; ++r) {
            if (!x.live(r)) continue;
            const uint32_t digit = (x.key[r] >> a.shift) & ((1u << a.bits) - 1u);
            const uint32_t at = whist[w * a.bins + digit] + x.rank[r];
            const uint32_t slot = FIRST ? x.at(r) : a.slot_in[x.at(r)];
            if (a.key_out) a.key_out[at] = x.key[r];
            if (a.slot_out) a.slot_out[at] = slot;
            if (a.position) a.position[slot] = (int32_t)at;
        }
        if (e - b0 <= block) break;  // the next block of the chunk
        b0 += block;
        __syncthreads();
        for (uint32_t i = t; i < kSortWaves * a.bins; i += kSortThreads) whist[i] = 0u;
        x.first = b0 + in_block;
#pragma unroll
        for (int r = 0; r < kItems; ++r) x.key[r] = x.live(r) ? sort_key<FIRST>(a, x.at(r)) : 0u;
        __syncthreads();
        rank_items(x, a.shift, a.bits, whist + w * a.bins);
        __syncthreads();
    }
}

// The place of an item is the number of items that go before it: those of a
// smaller key, and of the same key before it.  A workgroup places 16 items, each
// by 64 threads that go over n / 64 keys each (3000 ids 3.8 us; 32 items to a
// workgroup leave CUs idle, 4.6).  Further workgroups place the
// segments' borders in the same way: before offsets[s] go the keys below s.
constexpr uint32_t kRankItems = 16;
constexpr uint32_t kRankParts = kSortThreads / kRankItems;
// Keys that a thread goes over: whole blocks of 16.
__host__ __device__ inline uint32_t rank_part(uint32_t n) {
    return (n + kSortThreads - 1u) / kSortThreads * kRankItems;
}

// Workgroups that place items: one at least.
__host__ __device__ inline uint32_t rank_groups(uint32_t n) {
    return n ? (n + kRankItems - 1u) / kRankItems : 1u;
}

__global__ __launch_bounds__(kSortThreads) void rank_kernel(SortArgs a) {
    extern __shared__ uint4 staged[];  // twice each key; past the last one the largest number
    __shared__ uint32_t place[kRankItems];
    if (blockIdx.x >= a.chunks) return clear(a.fill, blockIdx.x - a.chunks, gridDim.x - a.chunks);
    uint32_t *const twice = reinterpret_cast<uint32_t *>(staged);
    const uint32_t t = threadIdx.x, items = rank_groups(a.n) * kRankItems;
    const bool borders = blockIdx.x * kRankItems >= items;
    // The chunk of the workgroup's items; `first` and `item` count from its start.
    const uint32_t base = borders ? 0u : blockIdx.x * kRankItems / a.chunk * a.chunk;
    const uint32_t count = min(a.chunk, a.n - base), first = blockIdx.x * kRankItems - base;
    const uint32_t per = rank_part(min(a.chunk, a.n)), all = per * kRankParts;
    for (uint32_t i = t; i < all; i += kSortThreads)
        twice[i] = i < count ? 2u * sort_key<true>(a, base + i) : 0xFFFFFFFFu;
    if (t < kRankItems) place[t] = 0u;
    __syncthreads();
    const uint32_t item = first + t % kRankItems, part = t / kRankItems;
    const uint32_t mine = borders ? 2u * (item - items) : item < count ? twice[item] : 0u;
    uint32_t before = 0;
    // A block of 16 keys lies before, at, or past the workgroup's items.  Before
    // them equal keys count: 2 key_j < 2 key_i + 1.
    for (uint32_t b = part * per; b < (part + 1u) * per; b += kRankItems) {
        const uint32_t limit = mine + (b < first && !borders ? 1u : 0u);
#pragma unroll
        for (uint32_t j = 0; j < kRankItems / 4; ++j) {
            const uint4 k = staged[b / 4 + j];
            before += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
        }
    }
    // Of the workgroup's own items, one each.
    const uint32_t other = first + part;
    if (!borders && part < kRankItems) before += other < item && twice[other] == mine;
    atomicAdd(&place[t % kRankItems], before);  // integers: any order gives the same sum
    __syncthreads();
    if (t >= kRankItems) return;
    const uint32_t at = base + place[t];
    if (borders) {
        if (item - items <= a.segments) a.offsets[item - items] = at;
    } else if (item < count) {
        if (a.key_out) a.key_out[at] = mine / 2u;
        if (a.slot_out) a.slot_out[at] = base + item;
        if (a.position) a.position[base + item] = (int32_t)at;
    }
}

// Chunks of 1024 items, each in order, joined: an item goes past its place in its
// own chunk by the keys of the other chunks that go before it, each found by
// halving.  A workgroup places 64 items (one to a lane), or 64 borders; its waves
// take the chunks in turn, 15 at a time from LDS.
constexpr uint32_t kMergeChunk = 1024, kMergeItems = 64, kMergeChunks = 15;

__global__ __launch_bounds__(kSortThreads) void merge_kernel(SortArgs a) {
    extern __shared__ uint4 staged[];  // keys; past the last one the largest number
    __shared__ uint32_t place[kMergeItems];
    if (blockIdx.x >= a.chunks) return clear(a.fill, blockIdx.x - a.chunks, gridDim.x - a.chunks);
    uint32_t *const keys = reinterpret_cast<uint32_t *>(staged);
    const uint32_t t = threadIdx.x, lane = t & 63u, w = t >> 6;
    const uint32_t items = (a.n + kMergeItems - 1u) / kMergeItems * kMergeItems;
    const uint32_t i = blockIdx.x * kMergeItems + lane;
    const bool borders = i >= items;
    const uint32_t key = borders ? i - items : i < a.n ? a.key_in[i] : 0u;
    const uint32_t own = borders ? 0xFFFFFFFFu : i / kMergeChunk;  // of the workgroup: 64 divides 1024
    const uint32_t chunks = (a.n + kMergeChunk - 1u) / kMergeChunk;
    if (t < kMergeItems) place[t] = 0u;
    uint32_t before = 0;
    for (uint32_t c0 = 0; c0 < chunks; c0 += kMergeChunks) {
        const uint32_t here = min(kMergeChunks, chunks - c0);
        __syncthreads();
        static_assert(kMergeChunk == kSortThreads, "a key of each chunk to a thread");
        uint32_t k[kMergeChunks];  // loaded together
#pragma unroll
        for (uint32_t j = 0; j < kMergeChunks; ++j) {
            const uint32_t at = (c0 + j) * kMergeChunk + t;
            k[j] = at < a.n ? a.key_in[at] : 0xFFFFFFFFu;
        }
#pragma unroll
        for (uint32_t j = 0; j < kMergeChunks; ++j)
            if (j < here) keys[j * kMergeChunk + t] = k[j];
        __syncthreads();
        if (w >= here) continue;
        const uint32_t c = c0 + w;
        if (c == own) {
            before += i % kMergeChunk;
            continue;
        }
        // Equal keys of an earlier chunk go before it.
        const uint32_t limit = key + (!borders && c < own ? 1u : 0u);
        const uint32_t *const list = keys + w * kMergeChunk;
        uint32_t below = 0;
#pragma unroll
        for (uint32_t step = kMergeChunk / 2; step; step >>= 1)
            if (list[below + step - 1u] < limit) below += step;
        before += below + (list[below] < limit ? 1u : 0u);
    }
    __syncthreads();
    if (before) atomicAdd(&place[lane], before);  // integers: any order gives the same sum
    __syncthreads();
    if (w) return;
    const uint32_t at = place[lane];
    if (borders) {
        if (key <= a.segments) a.offsets[key] = at;
    } else if (i < a.n) {
        const uint32_t slot = a.slot_in[i];
        if (a.key_out) a.key_out[at] = key;
        if (a.slot_out) a.slot_out[at] = slot;
        if (a.position) a.position[slot] = (int32_t)at;
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

// Counting against radix passes: among 128 segments (one pass) 5000 ids take 6.1 us
// against 7.4, 8000 8.8 against 7.5 but in one launch, of which each costs the host
// 2.2 to 2.8, 9000 13.5 against 7.8 (from about 6500 to 8192 ids, a captured graph,
// which does not pay the host, would be served better by radix).  Where radix takes
// two passes, four launches: 5000 among 3000 6.2 by counting, 7000 10.8 and 7.8 by
// chunks joined; with the search of 40001 borders 9000 take 17.9 by counting, 13.6
// by chunks and 22.3 by radix, 20000 18.6 and 23.1, 32768 among 131072 24.5 and 25.6,
// but then the tables of a gradient, cleared beside it, want the longer sort; 50000
// 40.8 and 28.1.  Borders past so many are searched in the sorted keys, in a launch
// of their own.
constexpr int64_t kMaxRanked = 5120, kMaxMerged = 20480, kMaxRankedOnePass = 8192;
constexpr int64_t kManyBorders = 4096;

struct SortPlan {
    bool ranked, merged;  // by rank_kernel alone, or with merge_kernel
    int passes, bits;
    uint32_t bins, chunk, chunks;
    size_t hist_bytes, pair_bytes, bytes;
};

SortPlan sort_plan(int64_t n, int64_t segments) {
    SortPlan p{};
    if (segments + 1 <= (int64_t)kMaxBins) {
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
    p.ranked = n <= (p.passes > 1 ? kMaxRanked : kMaxRankedOnePass);
    if (p.ranked) {
        p.chunks = rank_groups((uint32_t)n);
        p.pair_bytes = ((size_t)n * 4 + 255) & ~(size_t)255;
        p.bytes = p.passes > 1 ? p.pair_bytes : 0;
        return p;
    }
    if ((p.merged = p.passes > 1 && n <= kMaxMerged)) {
        p.chunks = rank_groups((uint32_t)n);
        p.pair_bytes = ((size_t)n * 4 + 255) & ~(size_t)255;
        p.bytes = 3 * p.pair_bytes;
        return p;
    }
    // Chunks of whole blocks (of part of one, where there are few items): few enough
    // for a workgroup to add up all their histograms, and more once that is little
    // next to a chunk.
    int64_t chunk = (n + 127) / 128;
    if (chunk > kBlock) chunk = (n + 255) / 256 > kBlock ? (n + 255) / 256 : kBlock;
    if (chunk < kMinChunk) chunk = kMinChunk;
    const int64_t unit = chunk > kBlock ? kBlock : kSortThreads;
    chunk = (chunk + unit - 1) / unit * unit;
    p.chunk = (uint32_t)chunk;
    p.chunks = (uint32_t)((n + chunk - 1) / chunk);
    p.hist_bytes = ((size_t)p.chunks * p.bins * 4 + 255) & ~(size_t)255;
    // Of a sort in several passes, the keys in order, where offsets are searched;
    // and keys and slots between the passes, in two buffers taken in turn.
    p.pair_bytes = ((size_t)n * 4 + 255) & ~(size_t)255;
    p.bytes = p.hist_bytes + (p.passes > 1 ? 5 : 0) * p.pair_bytes;
    return p;
}

}  // namespace

size_t sort_workspace(int64_t n, int64_t segments) { return sort_plan(n, segments).bytes; }

hipError_t queue_sort(const void *ids, int id_type, int64_t n, int64_t segments, int32_t *order,
                      int32_t *position, int64_t *offsets, uint32_t *sorted, void *workspace,
                      hipStream_t stream, const Fill *fill) {
    const SortPlan p = sort_plan(n, segments);
    char *ws = static_cast<char *>(workspace);
    uint32_t *pair[2][2] = {};
    if (p.passes > 1 && !sorted) sorted = reinterpret_cast<uint32_t *>(ws + p.hist_bytes);
    if (p.passes > 1 && !p.ranked)
        for (int i = 0; i < (p.merged ? 2 : 4); ++i)
            pair[i >> 1][i & 1] =
                reinterpret_cast<uint32_t *>(ws + p.hist_bytes + (i + 1) * p.pair_bytes);
    SortArgs a{};
    a.ids = ids;
    a.hist = reinterpret_cast<uint32_t *>(ws);
    a.n = (uint32_t)n;
    a.segments = (uint32_t)segments;
    a.chunk = p.ranked ? (n ? (uint32_t)n : 1u) : p.merged ? kMergeChunk : p.chunk;
    a.bins = p.bins;
    a.bits = (uint32_t)p.bits;
    a.wide = id_type == SEGTOPK_KEY_I64;
    const bool borders = (p.ranked || p.merged) && offsets && segments < kManyBorders;
    a.chunks = p.chunks + (borders && p.ranked ? (uint32_t)(segments / kRankItems + 1) : 0u);
    a.offsets = borders || p.passes == 1 ? offsets : nullptr;
    const Fill whole = fill ? *fill : Fill{};
    const uint64_t launches = p.ranked ? 1 : p.merged ? 2 : 2 * p.passes;
    const uint64_t share = ((whole.bytes + launches - 1) / launches + 15) & ~(uint64_t)15;
    uint64_t filled = 0;
    hipError_t err = hipSuccess;
    const auto queue = [&](auto kernel, size_t lds) {
        const uint64_t left = whole.bytes - filled;
        a.fill = whole;
        a.fill.data = static_cast<char *>(whole.data) + filled;
        a.fill.bytes = left < share ? left : share;
        filled += a.fill.bytes;
        err = launch(kernel, dim3(a.chunks + fill_blocks(a.fill, kSortThreads)), kSortThreads,
                     stream, lds, a);
        return err == hipSuccess;
    };
    if (p.ranked) {
        a.key_out = sorted;
        a.slot_out = reinterpret_cast<uint32_t *>(order);
        a.position = position;
        if (!queue(rank_kernel, (size_t)rank_part(a.n ? a.n : 1u) * kRankParts * 4)) return err;
    }
    if (p.merged) {
        a.key_out = pair[0][0];
        a.slot_out = pair[0][1];
        if (!queue(rank_kernel, (size_t)rank_part(kMergeChunk) * kRankParts * 4)) return err;
        a.key_in = a.key_out;
        a.slot_in = a.slot_out;
        a.key_out = sorted;
        a.slot_out = reinterpret_cast<uint32_t *>(order);
        a.position = position;
        a.chunks = (uint32_t)((n + kMergeItems - 1) / kMergeItems) +
                   (borders ? (uint32_t)(segments / kMergeItems + 1) : 0u);
        const int64_t held = (n + kMergeChunk - 1) / kMergeChunk;
        const size_t most = (size_t)(held < kMergeChunks ? held : kMergeChunks);
        if (!queue(merge_kernel, most * kMergeChunk * 4)) return err;
    }
    for (int i = 0; !p.ranked && !p.merged && i < p.passes; ++i) {
        const bool last = i == p.passes - 1;
        a.shift = (uint32_t)(i * p.bits);
        a.key_in = i ? pair[(i - 1) & 1][0] : nullptr;
        a.slot_in = i ? pair[(i - 1) & 1][1] : nullptr;
        a.key_out = last ? sorted : pair[i & 1][0];
        a.slot_out = last ? reinterpret_cast<uint32_t *>(order) : pair[i & 1][1];
        a.position = last ? position : nullptr;
        if (!queue(i ? count_kernel<false> : count_kernel<true>, 0)) return err;
        if (!queue(i ? scatter_kernel<false> : scatter_kernel<true>, 0)) return err;
    }
    if (offsets && !a.offsets)
        return launch(offsets_kernel, dim3((unsigned)((segments + 256) / 256)), 256, stream, 0,
                      sorted, (uint32_t)n, (uint32_t)segments, offsets);
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
