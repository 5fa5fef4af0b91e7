// Embedding lookup with scaling, and its gradient by sorted tokens.
//     y_i = scale table[token_i],     dtable_v = scale sum_{token_i = v} dy_i,
// rows whose token lies outside the table (padding, -1) are zero and add
// nothing.  Both are bound by HBM: the lookup reads the rows that occur and
// writes y; the gradient reads dy and writes the whole table.
//
// The gradient sorts the positions by token (stable, least significant digit
// first), so that a token's rows of dy stand together in the order of the
// batch: sums run in a fixed order, without atomics, and every table row is
// written once.
//
// Measured in graphs: the lookup of 262144 rows of 2048 in bf16, text-like
// tokens, 216 us (6.0 TB/s with each row that occurs counted once; some are read again
// from HBM).  The gradient of 131072 rows of 2048 to a table of 131072: 190
// us for 1.07 GB (159 at the measured copy's rate): sums and zeros 150, the sort 28, the long runs 11;
// of 1000 rows of 1360 in fp32 to 32003: 36 us (26), of which the sort takes 8.  One
// warp's or block's sum for each table row instead of segments: 514 us, the frequent tokens' blocks long behind the others.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "cpdr_internal.hpp"
#include "launch.cuh"
#include "vec_io.cuh"

namespace cpdr {
namespace {

using namespace vio;

constexpr int kThreads = 256, kWarps = kThreads / 32;

// A block's share of a matrix: `rows` rows from row0 on and `cols` 16-byte
// vectors of each from col0 on, which the threads walk through row by row.
struct Share {
    int64_t row0;
    int rows, col0, cols;
};
struct Split {
    int per_block;   // rows of a block
    int cols;        // vectors of a block
};
constexpr int kColVecs = 1024;   // vectors of a row in one block, at most

__device__ __forceinline__ Share share_of(const Split &s, int64_t rows, int vecs) {
    Share h;
    h.row0 = (int64_t)blockIdx.x * s.per_block;
    h.rows = (int)min((int64_t)s.per_block, rows - h.row0);
    h.col0 = blockIdx.y * s.cols;
    h.cols = min(s.cols, vecs - h.col0);
    return h;
}

// This thread's vectors of a share: (row, col) and how far the next one is.
struct Walk {
    int row, col, step_row, step_col, cols;
    __device__ __forceinline__ explicit Walk(const Share &h)
        : row(threadIdx.x / h.cols), col(threadIdx.x % h.cols), step_row(kThreads / h.cols), step_col(kThreads % h.cols),
          cols(h.cols) {}
    __device__ __forceinline__ void next() {
        row += step_row;
        col += step_col;
        if (col >= cols) {
            col -= cols;
            row++;
        }
    }
};

constexpr int kAhead = 4;   // vectors of a thread in flight

// ------------------------------------------------------------------ lookup
template <typename T>
__global__ void __launch_bounds__(kThreads)
embed_fwd_kernel(const int32_t *tokens, int64_t n, const T *table, int vocab, int width, float scale, T *y, Split split) {
    constexpr int V = kVecOf<T>;
    next_grid_may_start();
    previous_grid_done();
    const Share h = share_of(split, n, width / V);
    Walk w(h);
    while (w.row < h.rows) {
        int64_t to[kAhead];
        uint4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++, w.next()) {
            to[u] = -1;
            x[u] = make_uint4(0, 0, 0, 0);
            if (w.row >= h.rows) continue;
            const int64_t row = h.row0 + w.row;
            const int col = (h.col0 + w.col) * V, token = tokens[row];
            to[u] = row * width + col;
            if ((uint32_t)token < (uint32_t)vocab) x[u] = load16(table + (int64_t)token * width + col);
        }
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            if (to[u] < 0) continue;
            float f[V];
            widen16(x[u], f);
#pragma unroll
            for (int j = 0; j < V; j++) f[j] *= scale;
            // y is read by another kernel: it leaves the L2 to the table's rows (262144 x 2048: 221 -> 216 us)
            float4 r;
            store16(reinterpret_cast<T *>(&r), f);
            __stcs(reinterpret_cast<float4 *>(y + to[u]), r);
        }
    }
}

// ------------------------------------------------------------------ sort
// One pass orders the pairs (key, position) by up to kMaxBits bits of the key:
// from the counts of every tile's digits each block finds the places of its own
// pairs and moves them, each warp its own stretch; it counts the next pass's
// digits of the tiles that they go to.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 10, kMaxBins = 1 << kMaxBits;
constexpr int kPerLane = 8, kSub = kSortThreads * kPerLane;   // pairs that a block ranks at once
constexpr int kMaxTiles = 128, kMaxPasses = (31 + kMaxBits - 1) / kMaxBits;
constexpr int kOwnBins = kMaxBins / kSortThreads;              // digits of a thread
static_assert(kSub <= 65536 && 32 * kPerLane <= 65536, "a few pairs' positions and a warp's counts fit 16 bits");

struct Pass {
    const int32_t *tokens;
    const int2 *in;    // pairs (key, position); NULL: the first pass, which takes the tokens
    int2 *out;
    int32_t *counts;   // [passes][tiles][bins]
    int *longs;        // set to 0 for the sums
    int n, tile, tiles, vocab, pass, passes, bits;
    __device__ __forceinline__ int32_t *counts_of(int which) const { return counts + ((int64_t)which * tiles << bits); }
    // The key of position i: its token, or vocab (behind all others) where it lies outside the table.
    __device__ __forceinline__ int key_of(int i) const {
        const int k = tokens[i];
        return (uint32_t)k < (uint32_t)vocab ? k : vocab;
    }
};

// The ranks of keys (-1: none; `rounds` of them a lane) among those of their warp
// with the same digit, and in hist[warp][digit] how many there are.  The whole
// block calls it.
__device__ __forceinline__ void rank_keys(const int (&key)[kPerLane], int (&rank)[kPerLane], uint16_t (*hist)[kMaxBins],
                                          int rounds, int shift, int bits) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int d = lane; d < 1 << bits; d += 32) hist[w][d] = 0;
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        if (u >= rounds) break;
        const int digit = key[u] < 0 ? -1 : (key[u] >> shift) & ((1 << bits) - 1);
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        rank[u] = digit < 0 ? 0 : hist[w][digit] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (digit >= 0 && lane == 31 - __clz(same)) hist[w][digit] = (uint16_t)(rank[u] + 1);
        __syncwarp();
    }
    __syncthreads();
}

// place[d] = the sum of count[x] of the digits x before d; the whole block calls it.
__device__ __forceinline__ void places_of(const int *count, int *place, int bins, int *sums) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int c[kOwnBins], v = 0;
#pragma unroll
    for (int x = 0; x < kOwnBins; x++) {
        const int d = threadIdx.x * kOwnBins + x;
        c[x] = d < bins ? count[d] : 0;
        v += c[x];
    }
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) sums[w] = s;
    __syncthreads();
    s -= v;
#pragma unroll
    for (int i = 0; i < kSortWarps; i++)
        if (i < w) s += sums[i];
#pragma unroll
    for (int x = 0; x < kOwnBins; x++) {
        const int d = threadIdx.x * kOwnBins + x;
        if (d < bins) place[d] = s;
        s += c[x];
    }
    __syncthreads();
}

// The first pass's counts, and zeros for the others'.
__global__ void __launch_bounds__(kSortThreads) digit_counts_kernel(Pass p) {
    __shared__ int hist[kMaxBins];
    next_grid_may_start();
    const int bins = 1 << p.bits;
    for (int d = threadIdx.x; d < bins; d += kSortThreads) hist[d] = 0;
    __syncthreads();
    previous_grid_done();
    const int a = blockIdx.x * p.tile, b = min(p.n, a + p.tile);
    for (int i0 = a; i0 < b; i0 += kSub) {
        int key[kPerLane];
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            const int i = i0 + u * kSortThreads + threadIdx.x;
            key[u] = i < b ? p.key_of(i) : -1;
        }
#pragma unroll
        for (int u = 0; u < kPerLane; u++)
            if (key[u] >= 0) atomicAdd(&hist[key[u] & (bins - 1)], 1);   // a count has no order
    }
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) {
        const int64_t at = ((int64_t)blockIdx.x << p.bits) + d;
        p.counts[at] = hist[d];
        for (int i = 1; i < p.passes; i++) p.counts_of(i)[at] = 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.longs = 0;
}

__global__ void __launch_bounds__(kSortThreads) move_pairs_kernel(Pass p) {
    __shared__ uint16_t hist[kSortWarps][kMaxBins];
    __shared__ int place[kMaxBins], total[kMaxBins], sums[kSortWarps];
    next_grid_may_start();
    previous_grid_done();
    const int bins = 1 << p.bits;
    const int a = blockIdx.x * p.tile, b = min(p.n, a + p.tile), shift = p.pass * p.bits;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t *counts = p.counts_of(p.pass);
    int32_t *next_counts = p.pass + 1 < p.passes ? p.counts_of(p.pass + 1) : nullptr;
    int key[kPerLane], pos[kPerLane], rank[kPerLane];
    const int mine0 = w * 32 * kPerLane + lane;
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            const int i = i0 + mine0 + 32 * u;
            key[u] = -1;
            pos[u] = i;
            if (i >= b) continue;
            if (p.in) {
                const int2 x = p.in[i];
                key[u] = x.x;
                pos[u] = x.y;
            } else {
                key[u] = p.key_of(i);
            }
        }
    };
    load(a);
    // where this block's pairs of each digit go: behind all smaller digits and the blocks before
    int mine[kOwnBins];
#pragma unroll
    for (int x = 0; x < kOwnBins; x++) {
        const int d = x * kSortThreads + threadIdx.x;
        int all = 0;
        mine[x] = 0;
        if (d < bins) {
#pragma unroll 16
            for (int t = 0; t < p.tiles; t++) {
                const int c = counts[((int64_t)t << p.bits) + d];
                all += c;
                if (t < (int)blockIdx.x) mine[x] += c;
            }
            total[d] = all;
        }
    }
    __syncthreads();
    places_of(total, place, bins, sums);
#pragma unroll
    for (int x = 0; x < kOwnBins; x++) {
        const int d = x * kSortThreads + threadIdx.x;
        if (d < bins) place[d] += mine[x];
    }
    for (int i0 = a; i0 < b; i0 += kSub) {
        rank_keys(key, rank, hist, kPerLane, shift, p.bits);
        // hist becomes how many pairs of the digit the warps before have
        for (int d = threadIdx.x; d < bins; d += kSortThreads) {
            int before = 0;
#pragma unroll
            for (int x = 0; x < kSortWarps; x++) {
                const int c = hist[x][d];
                hist[x][d] = (uint16_t)before;
                before += c;
            }
            total[d] = before;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            if (key[u] < 0) continue;
            const int digit = (key[u] >> shift) & (bins - 1), at = place[digit] + hist[w][digit] + rank[u];
            p.out[at] = make_int2(key[u], pos[u]);
            if (next_counts) atomicAdd(&next_counts[((int64_t)(at / p.tile) << p.bits) + ((key[u] >> (shift + p.bits)) & (bins - 1))], 1);
        }
        if (i0 + kSub >= b) break;
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += kSortThreads) place[d] += total[d];
        __syncthreads();
        load(i0 + kSub);
    }
}

// All passes over at most kSub pairs, by one block.
__global__ void __launch_bounds__(kSortThreads) sort_few_kernel(Pass p) {
    __shared__ __align__(16) uint16_t hist[kSortWarps][kMaxBins];
    __shared__ int place[kMaxBins], sums[kSortWarps];
    // the pairs change places in the counts' memory
    static_assert(sizeof(hist) >= kSub * (sizeof(int) + sizeof(uint16_t)), "the pairs fit it");
    int *keys = (int *)&hist[0][0];
    uint16_t *places = (uint16_t *)(keys + kSub);
    next_grid_may_start();
    previous_grid_done();
    // every warp has a stretch of the list, of `rounds` pairs a lane
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = 1 << p.bits;
    const int rounds = (p.n + kSortThreads - 1) / kSortThreads, first = w * 32 * rounds + lane;
    int key[kPerLane], pos[kPerLane], rank[kPerLane];
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        pos[u] = first + 32 * u;
        key[u] = u < rounds && pos[u] < p.n ? p.key_of(pos[u]) : -1;
    }
    for (int i = 0; i < p.passes; i++) {
        const int shift = i * p.bits;
        rank_keys(key, rank, hist, rounds, shift, p.bits);
        for (int d = threadIdx.x; d < bins; d += kSortThreads) {
            int before = 0;
#pragma unroll
            for (int x = 0; x < kSortWarps; x++) {
                const int c = hist[x][d];
                hist[x][d] = (uint16_t)before;
                before += c;
            }
            place[d] = before;
        }
        __syncthreads();
        places_of(place, place, bins, sums);
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            if (key[u] < 0) continue;
            const int digit = (key[u] >> shift) & (bins - 1);
            rank[u] += place[digit] + hist[w][digit];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPerLane; u++)
            if (key[u] >= 0) {
                keys[rank[u]] = key[u];
                places[rank[u]] = (uint16_t)pos[u];
            }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            const int j = first + 32 * u;
            const bool mine = u < rounds && j < p.n;
            key[u] = mine ? keys[j] : -1;
            pos[u] = mine ? places[j] : 0;
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        const int j = first + 32 * u;
        if (u < rounds && j < p.n) p.out[j] = make_int2(key[u], pos[u]);
        if (j == 0) *p.longs = 0;
    }
}

// ------------------------------------------------------------------ sums
// The sorted list is cut into segments, so that a token in every place costs no
// more than one in few.  A segment sums the runs of one token that begin in it,
// to their ends, which may lie up to `beyond` pairs behind it.  A run that goes
// on further is long: each of its segments puts its part of the sum into `part`,
// and a second kernel adds those up.  Table rows that do not occur are
// filled by blocks of their own, among the segments'.
constexpr int kSegment = 32;   // a warp's lanes
// `beyond`, with so many segments that HBM bounds the sums, and with fewer, where
// the longest segment does: from 8 blocks of segments an SM on.  Text-like tokens, us with 128 and with 16, by
// blocks an SM: rows of 2048 at 1.7 119 and 111, at 3.4 134 and 127, at 5 141 and 142, at 6.7 144 and 149, at 8.4 155 and
// 163, at 13.5 190 and 202; rows of 256 at 1.3 80 and 55, at 3.4 96 and 79, at 6.7 138 and 130, at 10.3 194 and
// 192, at 13.5 220 and 222; rows of 64 at 13.5 179 and 164.  (It is by the sizes alone: where every token has runs of
// some 65, at 6.7 blocks, 128 takes 80 and 16 121.)
constexpr int kBeyondMany = 128, kBeyondFew = 16;
// Segments of a block, at most.  With 16 or 32: 100000 rows of 256 55 and 54 us, 262144 of 64 61 and 67, 1048576 of 64 164 and 156.
constexpr int kMaxGroups = 16;

struct Sums {
    const int2 *pair;           // (key, position), sorted
    const void *dy;
    void *dtable;
    int *longs;                 // how many long runs there are, and the segments that they begin in
    float *part;                // [segments][2][width]: a long run that comes from before, one that begins here
    int n, vocab, width;
    float scale;
    int beyond;
    int cols, groups;           // segments' blocks: vectors of a row (two for each thread), segments of a block
    int seg_blocks, zero_blocks, col_blocks;
    Split split;                // of the table, for the blocks that fill it
};

template <int V>
__device__ __forceinline__ void store_floats(float *to, const float (&x)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<float4 *>(to + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
}

// The whole warp calls it: the first pair whose key is not below k.
__device__ __forceinline__ int lower_bound(const int2 *pair, int n, int k) {
    const int lane = threadIdx.x & 31;
    int a = 0, len = n;   // it lies in a .. a + len
    while (len > 32) {
        const int step = len / 33, at = a + (lane + 1) * step;   // the last one: a + 32 (len / 33) < a + len
        const int below = __popc(__ballot_sync(0xffffffffu, pair[at].x < k));
        const int end = below < 32 ? a + (below + 1) * step : a + len;
        if (below) a += below * step + 1;
        len = end - a;
    }
    return a + __popc(__ballot_sync(0xffffffffu, lane < len && pair[a + lane].x < k));
}

constexpr int kTableRows = 512;   // table rows of a block, at most

// zeros in the rows of a share of the table that do not occur
template <typename T>
__device__ __forceinline__ void fill_rows(const Sums &p, const Share &h, uint32_t *occurs, int *ends) {
    for (int r = threadIdx.x; r < kTableRows / 32; r += kThreads) occurs[r] = 0;
    if (threadIdx.x < 64) {
        const int w = threadIdx.x >> 5, e = lower_bound(p.pair, p.n, (int)h.row0 + (w ? h.rows : 0));
        if ((threadIdx.x & 31) == 0) ends[w] = e;
    }
    __syncthreads();
    const int a = ends[0], b = ends[1];
    if (b - a <= 4 * kThreads) {
        for (int i = a + threadIdx.x; i < b; i += kThreads) {
            const int k = p.pair[i].x, r = k - (int)h.row0;
            if (i == a || p.pair[i - 1].x != k) atomicOr(&occurs[r >> 5], 1u << (r & 31));
        }
    } else {   // frequent tokens: a search for each row instead of a look at every pair
        for (int r = threadIdx.x; r < h.rows; r += kThreads) {
            const int k = (int)h.row0 + r;
            int lo = a, hi = b;
            while (lo < hi) {
                const int m = lo + (hi - lo) / 2;
                if (p.pair[m].x < k) lo = m + 1;
                else hi = m;
            }
            if (lo < b && p.pair[lo].x == k) atomicOr(&occurs[r >> 5], 1u << (r & 31));
        }
    }
    __syncthreads();
    T *to = (T *)p.dtable + h.row0 * p.width + h.col0 * kVecOf<T>;
    for (Walk w(h); w.row < h.rows; w.next())
        if (!(occurs[w.row >> 5] >> (w.row & 31) & 1))
            *reinterpret_cast<uint4 *>(to + (int64_t)w.row * p.width + w.col * kVecOf<T>) = make_uint4(0, 0, 0, 0);
}

// What a segment sums: pairs begin .. end - 1.
struct Plan {
    int begin, end;
    uint32_t ends;        // bit i: a run ends with the segment's pair i
    bool from_before;     // the first run is a long one, begun before
    bool goes_on;         // the last run is a long one, begun here
};

// The whole warp calls it; `pair` holds the segment's pairs.
__device__ __forceinline__ Plan plan_of(const Sums &p, const int2 *pair, int seg) {
    const int a = seg * kSegment, lane = threadIdx.x & 31;
    Plan s{a, a, 0, false, false};
    if (a >= p.n) return s;
    const int b = min(p.n, a + kSegment), len = b - a;
    const int key = pair[lane].x, first = pair[0].x, last = pair[len - 1].x;   // behind the list: vocab
    const uint32_t alike = __ballot_sync(0xffffffffu, lane < len && key == first);
    s.ends = __ballot_sync(0xffffffffu, lane + 1 < len && key != pair[lane + 1 < len ? lane + 1 : lane].x);
    const int tokens = __popc(__ballot_sync(0xffffffffu, key < p.vocab));   // padding stands last
    s.end = a + tokens;
    const int before = a ? p.pair[a - 1].x : -1, behind = b < p.n ? p.pair[b].x : -1;
    if (before == first && first < p.vocab) {
        // where it began, and whether it is long
        const int w0 = a - p.beyond - kSegment;
        bool is_long = w0 >= 0 && p.pair[w0 >= 0 ? w0 : 0].x == first;
        if (!is_long) {
            const int from = max(0, w0), start = from + lower_bound(p.pair + from, a - from, first);
            const int64_t limit = (int64_t)(start / kSegment + 1) * kSegment + p.beyond;
            is_long = limit < p.n && p.pair[limit].x == first;
        }
        s.from_before = is_long;
        if (!is_long) s.begin = a + __popc(alike);
    }
    if (behind == last && last < p.vocab && s.begin < b && !(s.from_before && last == first)) {
        const int64_t limit = (int64_t)b + p.beyond;
        s.goes_on = limit < p.n && p.pair[limit].x == last;
        if (!s.goes_on) s.end = b + lower_bound(p.pair + b, (int)min((int64_t)p.beyond, (int64_t)p.n - b), last + 1);
    }
    return s;
}

// Rows of dy on their way to a thread's places in shared memory, two vectors
// of each: 5 blocks of an SM have 160 KB in flight.
constexpr int kStages = 4;

// grid: the segments' and the filling blocks in turn
template <typename T>
__global__ void __launch_bounds__(kThreads, 5) segment_sums_kernel(Sums p) {
    constexpr int V = kVecOf<T>, H = V / 2;
    __shared__ uint4 stage[kStages][2][kThreads];   // each thread reads what it fetched itself
    __shared__ int2 pairs[kMaxGroups * kSegment];
    __shared__ Plan plans[kMaxGroups];
    __shared__ int ends[2];
    next_grid_may_start();
    previous_grid_done();
    // the roles alternate as long as there are blocks of both
    const int both_of = 2 * min(p.seg_blocks, p.zero_blocks), i = blockIdx.x;
    const bool fills = i < both_of ? i & 1 : p.seg_blocks < p.zero_blocks;
    const int at = i < both_of ? i >> 1 : i - both_of / 2;
    if (fills) {
        const int per_row = (p.width / V + p.split.cols - 1) / p.split.cols;
        Share h;
        h.row0 = (int64_t)(at / per_row) * p.split.per_block;
        h.rows = (int)min((int64_t)p.split.per_block, p.vocab - h.row0);
        h.col0 = at % per_row * p.split.cols;
        h.cols = min(p.split.cols, p.width / V - h.col0);
        fill_rows<T>(p, h, (uint32_t *)pairs, ends);
        return;
    }
    const int seg0 = at / p.col_blocks * p.groups;
    for (int x = threadIdx.x; x < p.groups * kSegment; x += kThreads) {
        const int j = seg0 * kSegment + x;
        pairs[x] = j < p.n ? p.pair[j] : make_int2(p.vocab, 0);
    }
    __syncthreads();
    for (int g = threadIdx.x >> 5; g < p.groups; g += kWarps) {
        const Plan s = plan_of(p, pairs + g * kSegment, seg0 + g);
        if ((threadIdx.x & 31) == 0) {
            plans[g] = s;
            // the list's order does not matter: every run is added up by itself
            if (s.goes_on && at % p.col_blocks == 0) p.longs[1 + atomicAdd(p.longs, 1)] = seg0 + g;
        }
    }
    __syncthreads();
    const int half = (p.cols + 1) / 2, group = threadIdx.x / half, mine = threadIdx.x % half;
    if (group >= p.groups) return;
    const int vec = at % p.col_blocks * p.cols + mine, vecs = p.width / V;
    if (vec >= vecs) return;
    const bool two = mine + half < p.cols && vec + half < vecs;   // the second vector is there
    const Plan s = plans[group];
    const int a = (seg0 + group) * kSegment;
    const int2 *pair = pairs + group * kSegment;
    const int col[2] = {vec * V, (two ? vec + half : vec) * V};
    const T *dy = (const T *)p.dy;
    auto fetch = [&](int j, int slot) {
        if (j < s.end) {
            const T *row = dy + (int64_t)(j < a + kSegment ? pair[j - a].y : p.pair[j].y) * p.width;
            fetch16(&stage[slot][0][threadIdx.x], row + col[0]);
            if (two) fetch16(&stage[slot][1][threadIdx.x], row + col[1]);
        }
        fetch_group();
    };
    float2 acc[2][H];
    auto clear = [&]() {
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
            for (int e = 0; e < H; e++) acc[c][e] = make_float2(0.f, 0.f);
    };
    clear();
    bool first = true;   // the segment's first run
    // a run is over, with pair j
    auto finish = [&](int j) {
        const bool before = first && s.from_before, on = s.goes_on && j == s.end - 1;
#pragma unroll
        for (int c = 0; c < 2; c++) {
            if (c && !two) continue;
            float f[V];
            const float scale = before || on ? 1.f : p.scale;
#pragma unroll
            for (int e = 0; e < H; e++) {
                f[2 * e] = acc[c][e].x * scale;
                f[2 * e + 1] = acc[c][e].y * scale;
            }
            if (before || on)
                store_floats(p.part + ((int64_t)(seg0 + group) * 2 + !before) * p.width + col[c], f);
            else
                store16((T *)p.dtable + (int64_t)pair[min(j - a, kSegment - 1)].x * p.width + col[c], f);
        }
        first = false;
        clear();
    };
#pragma unroll
    for (int u = 0; u < kStages; u++) fetch(s.begin + u, u);
#pragma unroll 1
    for (int j0 = s.begin; j0 < s.end; j0 += kStages) {
#pragma unroll
        for (int u = 0; u < kStages; u++) {
            const int j = j0 + u;
            if (j >= s.end) break;
            fetch_wait<kStages - 1>();
#pragma unroll
            for (int c = 0; c < 2; c++) {
                if (c && !two) continue;
                float2 f[H];
                widen_pairs(stage[u][c][threadIdx.x], f);
#pragma unroll
                for (int e = 0; e < H; e++) acc[c][e] = add2(acc[c][e], f[e]);
            }
            fetch(j + kStages, u);
            if (j == s.end - 1 || (j < a + kSegment && (s.ends >> (j - a) & 1))) finish(j);
        }
    }
    fetch_wait<0>();
}

// Four floats; volatile, so that a batch of loads stays ahead of the sums that
// take them (left to itself the compiler saves the registers: two loads in flight).
__device__ __forceinline__ float4 load_now(const float *p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ void add4(float4 &a, const float4 &b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}

// acc += the incoming runs of segments a .. b - 1, from column col on
__device__ __forceinline__ void add_parts(const Sums &p, int a, int b, int col, float4 &acc) {
    const int64_t row = 2 * (int64_t)p.width;
    const float *part = p.part + a * row + col;
    auto some = [&](auto count) {
        constexpr int N = decltype(count)::value;
        float4 x[N];
#pragma unroll
        for (int u = 0; u < N; u++) x[u] = load_now(part + u * row);
#pragma unroll
        for (int u = 0; u < N; u++) add4(acc, x[u]);
        part += N * row;
    };
#pragma unroll 1
    for (; a + 8 <= b; a += 8) some(std::integral_constant<int, 8>());
#pragma unroll 1
    for (; a < b; a++) some(std::integral_constant<int, 1>());
}

__device__ __forceinline__ void store_four(float *p, const float4 &v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store_four(__nv_bfloat16 *p, const float4 &v) {
    store2(p, make_float2(v.x, v.y));
    store2(p + 2, make_float2(v.z, v.w));
}

// The long runs, 128 columns at a time: the block's warps share a run's segments.
// grid: blocks that take the listed runs in turn
template <typename T>
__global__ void __launch_bounds__(kThreads) long_runs_kernel(Sums p) {
    __shared__ float4 sh[kWarps][32];
    next_grid_may_start();
    previous_grid_done();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col_blocks = (p.width + 127) / 128;
    const int64_t items = (int64_t)*p.longs * col_blocks;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int s = p.longs[1 + i / col_blocks], col = ((int)(i % col_blocks) * 32 + lane) * 4;
        const int k = p.pair[(int64_t)(s + 1) * kSegment - 1].x, m = (lower_bound(p.pair, p.n, k + 1) - 1) / kSegment - s;
        const int per = (m + kWarps - 1) / kWarps;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < p.width) {
            if (w == 0) acc = load_now(p.part + (2 * (int64_t)s + 1) * p.width + col);
            add_parts(p, s + 1 + min(m, w * per), s + 1 + min(m, (w + 1) * per), col, acc);
        }
        sh[w][lane] = acc;
        __syncthreads();
        if (w == 0 && col < p.width) {
#pragma unroll
            for (int y = 1; y < kWarps; y++) add4(acc, sh[y][lane]);
            store_four((T *)p.dtable + (int64_t)k * p.width + col,
                       make_float4(acc.x * p.scale, acc.y * p.scale, acc.z * p.scale, acc.w * p.scale));
        }
        __syncthreads();
    }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

int bits_of(int vocab) {   // keys are 0 .. vocab
    int bits = 1;
    while (bits < 31 && (vocab >> bits) != 0) bits++;
    return bits;
}

// Pairs of a block of the sort: one ranking's, or more where that makes more than kMaxTiles blocks.
int tile_of(int64_t n) {
    const int64_t most = (int64_t)kSub * kMaxTiles;
    return (int)(kSub * std::max<int64_t>(1, (n + most - 1) / most));
}

int64_t segments_of(int64_t n) { return (n + kSegment - 1) / kSegment; }

// The workspace: two lists of pairs, the passes' counts, the segments' sums.
struct Space {
    size_t list, counts, longs, part, bytes;
};
Space space(int64_t n, int width) {
    Space s{};
    s.list = round256((size_t)n * sizeof(int2));
    s.counts = (n > kSub ? 2 : 1) * s.list;
    s.longs = s.counts + (n > kSub ? (size_t)kMaxPasses * kMaxTiles * kMaxBins * 4 : 0);
    s.part = s.longs + round256((size_t)(1 + n / (kBeyondFew + 1)) * 4);
    s.bytes = s.part + (size_t)segments_of(n) * 2 * (size_t)width * 4;
    return s;
}

// Rows and vectors of a block: about `most` vectors, fewer where that leaves multiprocessors without a block.
Split split_of(int64_t rows, int vecs, int most, int max_rows, int sms) {
    Split s;
    s.cols = vecs <= kColVecs ? vecs : kColVecs;
    const int64_t full = std::max(1, std::min(max_rows, most / s.cols));
    const int64_t blocks_of_a_row = (vecs + s.cols - 1) / s.cols;
    s.per_block = (int)std::max<int64_t>(1, std::min(full, rows * blocks_of_a_row / (4 * sms)));
    return s;
}
dim3 grid_of(const Split &s, int64_t rows, int vecs) {
    return dim3((unsigned)((rows + s.per_block - 1) / s.per_block), (unsigned)((vecs + s.cols - 1) / s.cols));
}

constexpr int kBlockVecs = 4096;   // vectors of a block: 16 of each thread

template <typename T>
int backward(const int32_t *tokens, int n, int vocab, int width, float scale, const void *dy, void *dtable, char *ws,
             int sms, void *stream) {
    constexpr int V = kVecOf<T>;
    const Space s = space(n, width);
    int2 *list[2] = {(int2 *)ws, (int2 *)(ws + s.list)};
    const int bits = bits_of(vocab);
    Pass p{};
    p.tokens = tokens;
    p.out = list[0];
    p.counts = (int32_t *)(ws + s.counts);
    p.longs = (int *)(ws + s.longs);
    p.n = n;
    p.tile = tile_of(n);
    p.tiles = (n + p.tile - 1) / p.tile;
    p.vocab = vocab;
    p.passes = (bits + kMaxBits - 1) / kMaxBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    int rc = 0;
    if (n > 0 && n <= kSub) {
        rc = launch_early(sort_few_kernel, dim3(1), kSortThreads, 0, 1, stream, p);
    } else if (n > 0) {
        rc = launch_early(digit_counts_kernel, dim3((unsigned)p.tiles), kSortThreads, 0, 1, stream, p);
        for (; p.pass < p.passes && !rc; p.pass++) {
            p.out = list[p.pass & 1];
            rc = launch_early(move_pairs_kernel, dim3((unsigned)p.tiles), kSortThreads, 0, 1, stream, p);
            p.in = p.out;
        }
    }
    if (rc) return rc;
    const int vecs = width / V;
    Sums q{p.out, dy, dtable, p.longs, (float *)(ws + s.part), n, vocab, width, scale, 0};
    q.cols = std::min(vecs, 2 * kThreads);
    q.groups = std::min(kThreads / ((q.cols + 1) / 2), kMaxGroups);
    q.col_blocks = (vecs + q.cols - 1) / q.cols;
    const int64_t segments = segments_of(n), seg_blocks = (segments + q.groups - 1) / q.groups * q.col_blocks;
    q.beyond = seg_blocks >= 8 * sms ? kBeyondMany : kBeyondFew;
    q.split = split_of(vocab, vecs, kBlockVecs, kTableRows, sms);
    const dim3 fill = grid_of(q.split, vocab, vecs);
    const int64_t zero_blocks = (int64_t)fill.x * fill.y;
    if (seg_blocks + zero_blocks > 0x7fffffff) return (int)cudaErrorInvalidValue;
    q.seg_blocks = (int)seg_blocks;
    q.zero_blocks = (int)zero_blocks;
    rc = launch_early(segment_sums_kernel<T>, dim3((unsigned)(seg_blocks + zero_blocks)), kThreads, 0, 1, stream, q);
    if (rc || n <= kSegment + q.beyond) return rc;   // no run can be long
    // no more blocks than the longest possible list has items, and a wave of them
    const int64_t most = n / (q.beyond + 1) * ((width + 127) / 128);
    return launch_early(long_runs_kernel<T>, dim3((unsigned)std::min<int64_t>(most, 6 * sms)), kThreads, 0, 1, stream, q);
}

template <typename T>
int forward(const int32_t *tokens, int64_t n, const void *table, int vocab, int width, float scale, void *y, int sms,
            void *stream) {
    constexpr int V = kVecOf<T>;
    const Split s = split_of(n, width / V, kBlockVecs, kBlockVecs, sms);
    return launch_early(embed_fwd_kernel<T>, grid_of(s, n, width / V), kThreads, 0, 1, stream, tokens, n, (const T *)table, vocab,
                        width, scale, (T *)y, s);
}

}  // namespace

int launch_embed_fwd(const cpdr_ctx *c, const int32_t *tokens, int64_t n, const void *table, int vocab, int width,
                     float scale, void *y, void *stream) {
    if (n == 0) return 0;
    const int sms = device_sms(c->device);
    return c->plan.in_dtype == CPDR_DTYPE_F32
               ? forward<float>(tokens, n, table, vocab, width, scale, y, sms, stream)
               : forward<__nv_bfloat16>(tokens, n, table, vocab, width, scale, y, sms, stream);
}

size_t embed_bwd_workspace(int64_t n, int width) { return space(n, width).bytes; }

int launch_embed_bwd(const cpdr_ctx *c, const int32_t *tokens, int64_t n, int vocab, int width, float scale,
                     const void *dy, void *dtable, void *ws, void *stream) {
    const int sms = device_sms(c->device);
    return c->plan.in_dtype == CPDR_DTYPE_F32
               ? backward<float>(tokens, (int)n, vocab, width, scale, dy, dtable, (char *)ws, sms, stream)
               : backward<__nv_bfloat16>(tokens, (int)n, vocab, width, scale, dy, dtable, (char *)ws, sms, stream);
}

}  // namespace cpdr
