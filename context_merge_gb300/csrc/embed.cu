// Embedding lookup with scaling, and its gradient by sorted tokens.
//     y_i = scale table[token_i],     dtable_v = scale sum_{token_i = v} dy_i,
// rows whose token lies outside the table (padding, -1) are zero and add
// nothing.  Both are bound by HBM: the lookup reads the rows that occur and
// writes y; the gradient reads dy and writes the whole table.
//
// The gradient sorts the positions by token (stable, least significant digit
// first), so that a token's rows of dy stand together in the order of the
// batch: sums run in a fixed order, without atomics, and every table row is
// written once.  A token may stand in any share of the batch, so rows of the
// sorted list are first summed in 64s wherever a 64 holds one token only; a
// table row then adds fewer than 64 rows of dy at either end and the sums of
// the 64s between.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

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
            store16(y + to[u], f);
        }
    }
}

// ------------------------------------------------------------------ sort
// One pass orders the pairs (key, position) by up to kMaxBits bits of the key:
// blocks count the digits of their tiles, then every block finds the places of
// its own from all counts and moves its pairs, each warp its own stretch.
constexpr int kMaxBits = 10, kMaxBins = 1 << kMaxBits;
constexpr int kPerLane = 8, kSub = kThreads * kPerLane;   // pairs that a block ranks at once
constexpr int kMaxTiles = 128;
static_assert(kSub <= 65536, "a few pairs' positions fit 16 bits");
constexpr int kOwnBins = kMaxBins / kThreads;              // digits that a thread adds up

struct Pass {
    const int32_t *key, *pos;   // pos NULL: the first pass, whose keys are tokens
    int32_t *key_out, *pos_out;
    int32_t *counts;            // [tiles][bins]
    int n, tile, tiles, vocab, shift, bits;
};

// The key of pair i: its token, or vocab (behind all others) where it lies outside the table.
__device__ __forceinline__ int key_of(const Pass &p, int i) {
    const int k = p.key[i];
    return p.pos ? k : (uint32_t)k < (uint32_t)p.vocab ? k : p.vocab;
}

__device__ __forceinline__ void clear(int *x, int n) {
    for (int i = threadIdx.x; i < n; i += kThreads) x[i] = 0;
}

// The ranks of kSub keys (-1: none) among those of their warp with the same
// digit, and in hist[warp][digit] how many there are.
__device__ __forceinline__ void rank_keys(const int (&key)[kPerLane], int (&rank)[kPerLane], int (*hist)[kMaxBins], int shift, int bits) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        const int digit = key[u] < 0 ? -1 : (key[u] >> shift) & ((1 << bits) - 1);
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        rank[u] = digit < 0 ? 0 : hist[w][digit] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (digit >= 0 && lane == 31 - __clz(same)) hist[w][digit] = rank[u] + 1;
        __syncwarp();
    }
}

// v becomes the sum of the values of the threads before this one.
__device__ __forceinline__ int sum_before(int v, int *sums) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[w] = x;
    __syncthreads();
    int before = x - v;
#pragma unroll
    for (int i = 0; i < kWarps; i++)
        if (i < w) before += sums[i];
    return before;
}

__global__ void __launch_bounds__(kThreads) digit_counts_kernel(Pass p) {
    __shared__ int hist[kMaxBins];
    next_grid_may_start();
    clear(hist, 1 << p.bits);
    __syncthreads();
    previous_grid_done();
    const int a = blockIdx.x * p.tile, b = min(p.n, a + p.tile);
    for (int i0 = a; i0 < b; i0 += kSub) {
        int key[kPerLane];
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            const int i = i0 + u * kThreads + threadIdx.x;
            key[u] = i < b ? key_of(p, i) : -1;
        }
#pragma unroll
        for (int u = 0; u < kPerLane; u++)
            if (key[u] >= 0) atomicAdd(&hist[(key[u] >> p.shift) & ((1 << p.bits) - 1)], 1);   // a count has no order
    }
    __syncthreads();
    for (int d = threadIdx.x; d < 1 << p.bits; d += kThreads) p.counts[((int64_t)blockIdx.x << p.bits) + d] = hist[d];
}

__global__ void __launch_bounds__(kThreads) move_pairs_kernel(Pass p) {
    __shared__ int hist[kWarps][kMaxBins];
    __shared__ int place[kMaxBins];
    __shared__ int sums[kWarps];
    next_grid_may_start();
    previous_grid_done();
    // where this block's pairs of each digit go: behind all smaller digits and the blocks before
    const int bins = 1 << p.bits;
    {
        int all[kOwnBins], mine[kOwnBins], total = 0;
#pragma unroll
        for (int x = 0; x < kOwnBins; x++) {
            all[x] = mine[x] = 0;
            const int d = threadIdx.x * kOwnBins + x;
            if (d < bins) {
#pragma unroll 8
                for (int t = 0; t < p.tiles; t++) {
                    const int c = p.counts[((int64_t)t << p.bits) + d];
                    all[x] += c;
                    if (t < (int)blockIdx.x) mine[x] += c;
                }
            }
            total += all[x];
        }
        int before = sum_before(total, sums);
#pragma unroll
        for (int x = 0; x < kOwnBins; x++) {
            const int d = threadIdx.x * kOwnBins + x;
            if (d < bins) place[d] = before + mine[x];
            before += all[x];
        }
    }
    const int a = blockIdx.x * p.tile, b = min(p.n, a + p.tile);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i0 = a; i0 < b; i0 += kSub) {
        int key[kPerLane], rank[kPerLane];
        const int first = i0 + w * 32 * kPerLane + lane;
#pragma unroll
        for (int u = 0; u < kPerLane; u++) key[u] = first + 32 * u < b ? key_of(p, first + 32 * u) : -1;
        clear(&hist[0][0], kWarps * kMaxBins);
        __syncthreads();
        rank_keys(key, rank, hist, p.shift, p.bits);
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += kThreads) {
            int at = place[d];
#pragma unroll
            for (int x = 0; x < kWarps; x++) {
                const int c = hist[x][d];
                hist[x][d] = at;
                at += c;
            }
            place[d] = at;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            const int i = first + 32 * u;
            if (i >= b) continue;
            const int at = hist[w][(key[u] >> p.shift) & (bins - 1)] + rank[u];
            p.key_out[at] = key[u];
            p.pos_out[at] = p.pos ? p.pos[i] : i;
        }
        __syncthreads();
    }
}

// All passes over at most kSub pairs, by one block.
__global__ void __launch_bounds__(kThreads) sort_few_kernel(Pass p, int passes) {
    __shared__ int hist[kWarps][kMaxBins];
    __shared__ int sums[kWarps];
    __shared__ int keys[kSub];
    __shared__ uint16_t places[kSub];   // positions: below kSub
    next_grid_may_start();
    previous_grid_done();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, first = w * 32 * kPerLane + lane, bins = 1 << p.bits;
    int key[kPerLane], pos[kPerLane], rank[kPerLane];
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        pos[u] = first + 32 * u;
        key[u] = pos[u] < p.n ? key_of(p, pos[u]) : -1;
    }
    for (int i = 0; i < passes; i++) {
        const int shift = i * p.bits;
        clear(&hist[0][0], kWarps * kMaxBins);
        __syncthreads();
        rank_keys(key, rank, hist, shift, p.bits);
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int x = 0; x < kOwnBins; x++)
#pragma unroll
            for (int y = 0; y < kWarps; y++) total += hist[y][threadIdx.x * kOwnBins + x];
        int at = sum_before(total, sums);
#pragma unroll
        for (int x = 0; x < kOwnBins; x++)
#pragma unroll
            for (int y = 0; y < kWarps; y++) {
                int &c = hist[y][threadIdx.x * kOwnBins + x];
                const int here = c;
                c = at;
                at += here;
            }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPerLane; u++)
            if (key[u] >= 0) {
                const int to = hist[w][(key[u] >> shift) & (bins - 1)] + rank[u];
                keys[to] = key[u];
                places[to] = (uint16_t)pos[u];
            }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPerLane; u++) {
            const int j = first + 32 * u;
            key[u] = j < p.n ? keys[j] : -1;
            pos[u] = j < p.n ? places[j] : 0;
        }
    }
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        const int j = first + 32 * u;
        if (j < p.n) {
            p.key_out[j] = key[u];
            p.pos_out[j] = pos[u];
        }
    }
}

// ------------------------------------------------------------------ sums
constexpr int kRun = 64;   // sorted pairs, or sums of such, that are summed ahead where they hold one token

struct Sums {
    const int32_t *key, *pos;   // sorted
    const void *dy;
    void *dtable;
    float *part, *part2;        // sums of whole runs of kRun pairs, and of kRun such runs: [.., width]
    int n, vocab, width;
    float scale;
    Split split;
};

template <int V>
__device__ __forceinline__ void add(float (&acc)[V], const uint4 &raw) {
    float x[V];
    widen16(raw, x);
#pragma unroll
    for (int j = 0; j < V; j++) acc[j] += x[j];
}

// acc += rows pos[a .. b) of dy, from column col on
template <typename T, int V>
__device__ __forceinline__ void add_rows(const Sums &p, int a, int b, int col, float (&acc)[V]) {
    const T *dy = (const T *)p.dy + col;
    for (; a < b; a += kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++)
            x[u] = a + u < b ? load16(dy + (int64_t)p.pos[a + u] * p.width) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < kAhead; u++) add<V>(acc, x[u]);
    }
}

// acc += rows a .. b - 1 of part, from column col on
template <int V>
__device__ __forceinline__ void add_sums(const float *part, int width, int a, int b, int col, float (&acc)[V]) {
    part += (int64_t)a * width + col;
    for (; a < b; a += kAhead, part += (int64_t)kAhead * width) {
        float4 x[kAhead][V / 4];
#pragma unroll
        for (int u = 0; u < kAhead; u++)
#pragma unroll
            for (int j = 0; j < V / 4; j++)
                x[u][j] = a + u < b ? *reinterpret_cast<const float4 *>(part + (int64_t)u * width + 4 * j)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kAhead; u++)
#pragma unroll
            for (int j = 0; j < V / 4; j++) {
                acc[4 * j] += x[u][j].x;
                acc[4 * j + 1] += x[u][j].y;
                acc[4 * j + 2] += x[u][j].z;
                acc[4 * j + 3] += x[u][j].w;
            }
    }
}

// SECOND: of kRun runs' sums.  grid (whole runs, blocks of columns)
template <typename T, bool SECOND>
__global__ void __launch_bounds__(kThreads) run_sums_kernel(Sums p) {
    constexpr int V = kVecOf<T>, LEN = SECOND ? kRun * kRun : kRun;
    next_grid_may_start();
    previous_grid_done();
    const int a = blockIdx.x * LEN, col = (blockIdx.y * kThreads + threadIdx.x) * V;
    const int k = p.key[a];
    if (k != p.key[a + LEN - 1] || k >= p.vocab || col >= p.width) return;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; j++) acc[j] = 0.f;
    if (SECOND) add_sums<V>(p.part, p.width, a / kRun, a / kRun + kRun, col, acc);
    else add_rows<T, V>(p, a, a + LEN, col, acc);
    float *to = (SECOND ? p.part2 : p.part) + (int64_t)blockIdx.x * p.width + col;
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<float4 *>(to + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
}

// The whole warp calls it: the first pair whose key is not below k.
__device__ __forceinline__ int lower_bound(const int32_t *key, int n, int k) {
    const int lane = threadIdx.x & 31;
    int a = 0, len = n;   // it lies in a .. a + len
    while (len > 32) {
        const int step = len / 33, at = a + (lane + 1) * step;   // the last one: a + 32 (len / 33) < a + len
        const int below = __popc(__ballot_sync(0xffffffffu, key[at] < k));
        const int end = below < 32 ? a + (below + 1) * step : a + len;
        if (below) a += below * step + 1;
        len = end - a;
    }
    return a + __popc(__ballot_sync(0xffffffffu, lane < len && key[a + (lane < len ? lane : 0)] < k));
}

constexpr int kTableRows = 256;   // table rows of a block, at most

// acc += the sum of pairs a .. b - 1 of the sorted list, which hold one token
template <typename T, int V>
__device__ __forceinline__ void add_pairs(const Sums &p, int a, int b, int col, float (&acc)[V]) {
    const int c0 = (a + kRun - 1) / kRun, c1 = b / kRun;   // whole runs
    if (c0 >= c1) {
        add_rows<T, V>(p, a, b, col, acc);
        return;
    }
    add_rows<T, V>(p, a, c0 * kRun, col, acc);
    const int d0 = (c0 + kRun - 1) / kRun, d1 = c1 / kRun;
    if (d0 >= d1) {
        add_sums<V>(p.part, p.width, c0, c1, col, acc);
    } else {
        add_sums<V>(p.part, p.width, c0, d0 * kRun, col, acc);
        add_sums<V>(p.part2, p.width, d0, d1, col, acc);
        add_sums<V>(p.part, p.width, d1 * kRun, c1, col, acc);
    }
    add_rows<T, V>(p, c1 * kRun, b, col, acc);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) table_rows_kernel(Sums p) {
    constexpr int V = kVecOf<T>;
    __shared__ int first[kTableRows], last[kTableRows], ends[2];   // pairs of each row: first .. last - 1
    next_grid_may_start();
    previous_grid_done();
    const Share h = share_of(p.split, p.vocab, p.width / V);
    for (int r = threadIdx.x; r < h.rows; r += kThreads) first[r] = last[r] = 0;
    if (threadIdx.x < 64) {
        const int w = threadIdx.x >> 5, e = lower_bound(p.key, p.n, (int)h.row0 + (w ? h.rows : 0));
        if ((threadIdx.x & 31) == 0) ends[w] = e;
    }
    __syncthreads();
    const int a = ends[0], b = ends[1];
    for (int i = a + threadIdx.x; i < b; i += kThreads) {
        const int k = p.key[i], r = k - (int)h.row0;
        if (i == a || p.key[i - 1] != k) first[r] = i;
        if (i == b - 1 || p.key[i + 1] != k) last[r] = i + 1;
    }
    __syncthreads();
    Walk w(h);
    while (w.row < h.rows) {
        int row[kAhead], col[kAhead];
        uint4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++, w.next()) {
            row[u] = w.row;
            col[u] = (h.col0 + w.col) * V;
            x[u] = make_uint4(0, 0, 0, 0);
            if (row[u] < h.rows && last[row[u]] != 0)
                x[u] = load16((const T *)p.dy + (int64_t)p.pos[first[row[u]]] * p.width + col[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            if (row[u] >= h.rows) continue;
            const int i = first[row[u]], e = last[row[u]];
            float acc[V];
            widen16(x[u], acc);
            if (e > i + 1) {
                // whole runs start at the first pair: it is not taken by itself
                if (e - i >= kRun) {
#pragma unroll
                    for (int j = 0; j < V; j++) acc[j] = 0.f;
                    add_pairs<T, V>(p, i, e, col[u], acc);
                } else {
                    add_rows<T, V>(p, i + 1, e, col[u], acc);
                }
            }
#pragma unroll
            for (int j = 0; j < V; j++) acc[j] *= p.scale;
            store16((T *)p.dtable + (h.row0 + row[u]) * p.width + col[u], acc);
        }
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
    return (int)(kSub * ((n + most - 1) / most));
}

// The workspace: two lists of keys and positions, the counts, the runs' sums.
struct Space {
    size_t list, counts, part, part2, bytes;
};
Space space(int64_t n, int width) {
    Space s{};
    s.list = round256((size_t)n * 4);
    s.counts = 4 * s.list;
    s.part = s.counts + (n > kSub ? (size_t)kMaxTiles * kMaxBins * 4 : 0);
    s.part2 = s.part + (size_t)(n / kRun) * (size_t)width * 4;
    s.bytes = s.part2 + (size_t)(n / (kRun * kRun)) * (size_t)width * 4;
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
    int32_t *key[2] = {(int32_t *)ws, (int32_t *)(ws + s.list)};
    int32_t *pos[2] = {(int32_t *)(ws + 2 * s.list), (int32_t *)(ws + 3 * s.list)};
    const int bits = bits_of(vocab), passes = (bits + kMaxBits - 1) / kMaxBits;
    Pass p{};
    p.key = tokens;
    p.key_out = key[0];
    p.pos_out = pos[0];
    p.counts = (int32_t *)(ws + s.counts);
    p.n = n;
    p.tile = tile_of(n);
    p.vocab = vocab;
    p.bits = (bits + passes - 1) / passes;
    int rc = 0;
    if (n > 0 && n <= kSub) {
        rc = launch_early(sort_few_kernel, dim3(1), kThreads, 0, 1, stream, p, passes);
        p.key = key[0];
        p.pos = pos[0];
    } else if (n > 0) {
        p.tiles = (n + p.tile - 1) / p.tile;
        for (int i = 0; i < passes && !rc; i++, p.shift += p.bits) {
            p.key_out = key[i & 1];
            p.pos_out = pos[i & 1];
            rc = launch_early(digit_counts_kernel, dim3((unsigned)p.tiles), kThreads, 0, 1, stream, p);
            if (!rc) rc = launch_early(move_pairs_kernel, dim3((unsigned)p.tiles), kThreads, 0, 1, stream, p);
            p.key = p.key_out;
            p.pos = p.pos_out;
        }
    }
    if (rc) return rc;
    Sums q{p.key, p.pos, dy, dtable, (float *)(ws + s.part), (float *)(ws + s.part2), n, vocab, width, scale, {}};
    const unsigned cols = (unsigned)((width + kThreads * V - 1) / (kThreads * V));
    if (n >= kRun) rc = launch_early(run_sums_kernel<T, false>, dim3((unsigned)(n / kRun), cols), kThreads, 0, 1, stream, q);
    if (!rc && n >= kRun * kRun)
        rc = launch_early(run_sums_kernel<T, true>, dim3((unsigned)(n / (kRun * kRun)), cols), kThreads, 0, 1, stream, q);
    if (rc) return rc;
    q.split = split_of(vocab, width / V, kBlockVecs, kTableRows, sms);
    return launch_early(table_rows_kernel<T>, grid_of(q.split, vocab, width / V), kThreads, 0, 1, stream, q);
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
