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

// ------------------------------------------------------------------ lookup
// grid (rows, blocks of columns)
template <typename T>
__global__ void __launch_bounds__(kThreads)
embed_fwd_kernel(const int32_t *tokens, const T *table, int vocab, int width, float scale, T *y) {
    constexpr int V = kVecOf<T>;
    next_grid_may_start();
    previous_grid_done();
    const int64_t row = blockIdx.x;
    const int col = (blockIdx.y * kThreads + threadIdx.x) * V;
    if (col >= width) return;
    const int token = tokens[row];
    float x[V];
    widen16((uint32_t)token < (uint32_t)vocab ? load16(table + (int64_t)token * width + col) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
    for (int j = 0; j < V; j++) x[j] *= scale;
    store16(y + row * width + col, x);
}

// ------------------------------------------------------------------ sort
// One pass orders the pairs (key, position) by kBits bits of the key: blocks
// count the digits of their tiles, one block turns the counts into places,
// and every block moves its pairs, each warp its own stretch of the tile.
constexpr int kBits = 8, kBins = 1 << kBits;
constexpr int kPerLane = 8, kTile = kThreads * kPerLane;

struct Pass {
    const int32_t *key, *pos;   // pos NULL: the first pass, whose keys are tokens
    int32_t *key_out, *pos_out;
    int32_t *counts;            // [kBins][tiles]
    int n, tiles, vocab, shift;
};

// The key of pair i: its token, or vocab (behind all others) where it lies outside the table.
__device__ __forceinline__ int key_of(const Pass &p, int i) {
    const int k = p.key[i];
    return p.pos ? k : (uint32_t)k < (uint32_t)p.vocab ? k : p.vocab;
}

// Counts of each warp's digits in `hist`, and of this lane's pairs before it: in[u].
__device__ __forceinline__ void rank_tile(const Pass &p, int (*hist)[kBins], int (&key)[kPerLane], int (&rank)[kPerLane]) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kWarps * kBins; i += kThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    const int first = blockIdx.x * kTile + w * 32 * kPerLane + lane;
#pragma unroll
    for (int u = 0; u < kPerLane; u++) key[u] = first + 32 * u < p.n ? key_of(p, first + 32 * u) : -1;
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        const int digit = key[u] < 0 ? -1 : (key[u] >> p.shift) & (kBins - 1);
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        const int before = digit < 0 ? 0 : hist[w][digit];
        rank[u] = before + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (digit >= 0 && lane == 31 - __clz(same)) hist[w][digit] = rank[u] + 1;
        __syncwarp();
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads) digit_counts_kernel(Pass p) {
    __shared__ int hist[kWarps][kBins];
    next_grid_may_start();
    previous_grid_done();
    int key[kPerLane], rank[kPerLane];
    rank_tile(p, hist, key, rank);
    for (int d = threadIdx.x; d < kBins; d += kThreads) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) sum += hist[w][d];
        p.counts[(int64_t)d * p.tiles + blockIdx.x] = sum;
    }
}

constexpr int kScanThreads = 1024;

// counts[i] <- sum of counts before i: one block, each thread a stretch of its own.
__global__ void __launch_bounds__(kScanThreads) places_kernel(int32_t *counts, int total) {
    __shared__ int sums[32];
    next_grid_may_start();
    previous_grid_done();
    const int per = (total + kScanThreads - 1) / kScanThreads, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int a = min(total, (int)threadIdx.x * per), b = min(total, a + per);
    int sum = 0;
    for (int i = a; i < b; i++) sum += counts[i];
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[w] = x;
    __syncthreads();
    if (w == 0) {
        int s = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        sums[lane] = s;
    }
    __syncthreads();
    int before = x - sum + (w ? sums[w - 1] : 0);
    for (int i = a; i < b; i++) {
        const int c = counts[i];
        counts[i] = before;
        before += c;
    }
}

__global__ void __launch_bounds__(kThreads) move_pairs_kernel(Pass p) {
    __shared__ int hist[kWarps][kBins];
    next_grid_may_start();
    previous_grid_done();
    int key[kPerLane], rank[kPerLane];
    rank_tile(p, hist, key, rank);
    // from counts of each warp to the place of its first pair of each digit
    for (int d = threadIdx.x; d < kBins; d += kThreads) {
        int place = p.counts[(int64_t)d * p.tiles + blockIdx.x];
        for (int w = 0; w < kWarps; w++) {
            const int c = hist[w][d];
            hist[w][d] = place;
            place += c;
        }
    }
    __syncthreads();
    const int w = threadIdx.x >> 5, first = blockIdx.x * kTile + w * 32 * kPerLane + (threadIdx.x & 31);
#pragma unroll
    for (int u = 0; u < kPerLane; u++) {
        const int i = first + 32 * u;
        if (i >= p.n) continue;
        const int at = hist[w][(key[u] >> p.shift) & (kBins - 1)] + rank[u];
        p.key_out[at] = key[u];
        p.pos_out[at] = p.pos ? p.pos[i] : i;
    }
}

// ------------------------------------------------------------------ sums
constexpr int kRun = 64;   // sorted pairs that are summed ahead where they hold one token

struct Sums {
    const int32_t *key, *pos;   // sorted
    const void *dy;
    void *dtable;
    float *part;                // [n / kRun, width]
    int n, vocab, width;
    float scale;
};

// acc += rows pos[a .. b) of dy, from column col on
template <typename T, int V>
__device__ __forceinline__ void add_rows(const Sums &p, int a, int b, int col, float (&acc)[V]) {
    const T *dy = (const T *)p.dy;
    for (int i = a; i < b; i++) {
        float x[V];
        widen16(load16(dy + (int64_t)p.pos[i] * p.width + col), x);
#pragma unroll
        for (int j = 0; j < V; j++) acc[j] += x[j];
    }
}

// grid (whole runs of kRun pairs, blocks of columns)
template <typename T>
__global__ void __launch_bounds__(kThreads) run_sums_kernel(Sums p) {
    constexpr int V = kVecOf<T>;
    next_grid_may_start();
    previous_grid_done();
    const int a = blockIdx.x * kRun, col = (blockIdx.y * kThreads + threadIdx.x) * V;
    const int k = p.key[a];
    if (k != p.key[a + kRun - 1] || k >= p.vocab || col >= p.width) return;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; j++) acc[j] = 0.f;
    add_rows<T>(p, a, a + kRun, col, acc);
#pragma unroll
    for (int j = 0; j < V; j += 4)
        *reinterpret_cast<float4 *>(p.part + (int64_t)blockIdx.x * p.width + col + j) =
            make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
}

// The first pair whose key is not below k.
__device__ __forceinline__ int lower_bound(const int32_t *key, int n, int k) {
    int a = 0, b = n;
    while (a < b) {
        const int m = (int)(((int64_t)a + b) / 2);
        if (key[m] < k) a = m + 1;
        else b = m;
    }
    return a;
}

constexpr int kTableRows = 16;   // table rows of a block

// grid (blocks of table rows, blocks of columns)
template <typename T>
__global__ void __launch_bounds__(kThreads) table_rows_kernel(Sums p) {
    constexpr int V = kVecOf<T>;
    __shared__ int start[kTableRows + 1];
    next_grid_may_start();
    previous_grid_done();
    const int v0 = blockIdx.x * kTableRows, rows = min(kTableRows, p.vocab - v0);
    if (threadIdx.x <= rows) start[threadIdx.x] = lower_bound(p.key, p.n, v0 + threadIdx.x);
    __syncthreads();
    const int col = (blockIdx.y * kThreads + threadIdx.x) * V;
    if (col >= p.width) return;
    for (int r = 0; r < rows; r++) {
        const int a = start[r], b = start[r + 1];
        // whole runs c0 .. c1 - 1 of this token, if any
        const int c0 = (a + kRun - 1) / kRun, c1 = b / kRun;
        float acc[V];
#pragma unroll
        for (int j = 0; j < V; j++) acc[j] = 0.f;
        if (c0 >= c1) {
            add_rows<T>(p, a, b, col, acc);
        } else {
            add_rows<T>(p, a, c0 * kRun, col, acc);
            for (int c = c0; c < c1; c++)
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(p.part + (int64_t)c * p.width + col + j);
                    acc[j] += x.x;
                    acc[j + 1] += x.y;
                    acc[j + 2] += x.z;
                    acc[j + 3] += x.w;
                }
            add_rows<T>(p, c1 * kRun, b, col, acc);
        }
#pragma unroll
        for (int j = 0; j < V; j++) acc[j] *= p.scale;
        store16((T *)p.dtable + (int64_t)(v0 + r) * p.width + col, acc);
    }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

int passes_of(int vocab) {   // keys are 0 .. vocab
    int bits = 1;
    while (bits < 31 && (vocab >> bits) != 0) bits++;
    return (bits + kBits - 1) / kBits;
}

// The workspace: two lists of keys and positions, the counts, the runs' sums.
struct Space {
    size_t list, counts, part, bytes;
};
Space space(int64_t n, int width) {
    Space s{};
    s.list = round256((size_t)n * 4);
    s.counts = 4 * s.list;
    s.part = s.counts + round256((size_t)((n + kTile - 1) / kTile) * kBins * 4);
    s.bytes = s.part + (size_t)(n / kRun) * (size_t)width * 4;
    return s;
}

template <typename T>
int backward(const int32_t *tokens, int n, int vocab, int width, float scale, const void *dy, void *dtable, char *ws,
             void *stream) {
    const Space s = space(n, width);
    int32_t *key[2] = {(int32_t *)ws, (int32_t *)(ws + s.list)};
    int32_t *pos[2] = {(int32_t *)(ws + 2 * s.list), (int32_t *)(ws + 3 * s.list)};
    Pass p{tokens, nullptr, nullptr, nullptr, (int32_t *)(ws + s.counts), n, (n + kTile - 1) / kTile, vocab, 0};
    const int passes = n ? passes_of(vocab) : 0;
    for (int i = 0; i < passes; i++, p.shift += kBits) {
        p.key_out = key[i & 1];
        p.pos_out = pos[i & 1];
        int rc = launch_early(digit_counts_kernel, dim3((unsigned)p.tiles), kThreads, 0, 1, stream, p);
        if (!rc) rc = launch_early(places_kernel, dim3(1), kScanThreads, 0, 1, stream, p.counts, p.tiles * kBins);
        if (!rc) rc = launch_early(move_pairs_kernel, dim3((unsigned)p.tiles), kThreads, 0, 1, stream, p);
        if (rc) return rc;
        p.key = p.key_out;
        p.pos = p.pos_out;
    }
    const Sums q{p.key, p.pos, dy, dtable, (float *)(ws + s.part), n, vocab, width, scale};
    const unsigned cols = (unsigned)((width + kThreads * kVecOf<T> - 1) / (kThreads * kVecOf<T>));
    if (n >= kRun) {
        const int rc = launch_early(run_sums_kernel<T>, dim3((unsigned)(n / kRun), cols), kThreads, 0, 1, stream, q);
        if (rc) return rc;
    }
    return launch_early(table_rows_kernel<T>, dim3((unsigned)((vocab + kTableRows - 1) / kTableRows), cols), kThreads, 0, 1, stream, q);
}

}  // namespace

int launch_embed_fwd(const cpdr_ctx *c, const int32_t *tokens, int64_t n, const void *table, int vocab, int width,
                     float scale, void *y, void *stream) {
    if (n == 0) return 0;
    if (c->plan.in_dtype == CPDR_DTYPE_F32) {
        const dim3 grid((unsigned)n, (unsigned)((width + kThreads * 4 - 1) / (kThreads * 4)));
        return launch_early(embed_fwd_kernel<float>, grid, kThreads, 0, 1, stream, tokens, (const float *)table, vocab, width,
                            scale, (float *)y);
    }
    const dim3 grid((unsigned)n, (unsigned)((width + kThreads * 8 - 1) / (kThreads * 8)));
    return launch_early(embed_fwd_kernel<__nv_bfloat16>, grid, kThreads, 0, 1, stream, tokens, (const __nv_bfloat16 *)table,
                        vocab, width, scale, (__nv_bfloat16 *)y);
}

size_t embed_bwd_workspace(int64_t n, int width) { return space(n, width).bytes; }

int launch_embed_bwd(const cpdr_ctx *c, const int32_t *tokens, int64_t n, int vocab, int width, float scale,
                     const void *dy, void *dtable, void *ws, void *stream) {
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        return backward<float>(tokens, (int)n, vocab, width, scale, dy, dtable, (char *)ws, stream);
    return backward<__nv_bfloat16>(tokens, (int)n, vocab, width, scale, dy, dtable, (char *)ws, stream);
}

}  // namespace cpdr
