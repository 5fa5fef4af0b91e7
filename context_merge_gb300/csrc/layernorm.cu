// Layer norm with the residual's addition, and its gradients.  Per row of
// `width` elements, with s = x + residual (or x),
//     m = mean(s),   rstd = 1 / sqrt(mean((s - m)^2) + eps),
//     y_i = (s_i - m) rstd w_i + b_i,
// as T (fp32 or bf16), or as e4m3 with one scale per row,
//     scale = max(max_i |y_i| / 448, 2^-126),   y8_i = e4m3(y_i (1 / scale));
// backward, with xh = (s - m) rstd and u = w dy, from dy and (optionally) the
// gradient dsum that reaches s by the residual stream,
//     ds_i = rstd (u_i - mean(u) - xh_i mean(u xh)) + dsum_i,
//     dw_i = sum over rows of dy_i xh_i,   db_i = sum over rows of dy_i.
//
// Bound by HBM: every tensor is read and written once; a row lives in the
// registers of one group of threads.  The variance is summed from differences
// to a mean, which a row with a large mean needs: each warp takes its own
// columns' mean first and the sums of the differences to it then, without leaving
// the warp, and one exchange between warps joins them: with a_v the mean of warp
// v and A that of all,
//     sum (s - A)^2 = sum over v of  sum_v (s - a_v)^2 + n_v (a_v - A)^2
// (and the same for sum u (s - A)).  A fp32 mean is itself off by some half steps
// of the row's size; the sum of the differences says by how much, and what
// is subtracted is corrected by it.
//
// Measured over 0.25 GB a tensor, TB/s (the measured copy: 6.8): forward with a
// residual 6.4 to 7.0 at 64 to 16384 columns of bf16 and 6.2 to 7.0 of fp32;
// without one 5.0 to 6.4 (bf16, up to 4096; 3.7 to 5.0 beyond) and 6.3 to 6.9 (fp32);
// to e4m3 from bf16 5.2 to 6.8 up to 4096 and 3.8 to 5.5 beyond; backward with the
// residual's gradient 5.4 to 6.8 (bf16 up to 4096 columns, but 4.6 at 776; 3.1 to 5.4
// beyond) and 5.9 to 6.9 (fp32 up to 6144; 4.1 to 5.6 beyond).  What is below the
// copy's rate is bound by the exchanges up to 4096 columns: rows of bf16 have half the
// bytes for them.  Wide rows: forward, a row's loads are not on their way during the
// exchanges of the one before (three and four vectors a thread do not stream), and
// beyond 8192 columns of bf16 one block fills an SM; backward, beyond 12288 columns of
// bf16 and 6144 of fp32 there is room for one stage alone, so that loads and arithmetic
// take turns, the forms of bf16 with 512 x 3 and 512 x 4 and of fp32 with 512 x 8 spill
// 132, 464 and 288 bytes a thread, and fp32 rows beyond 8192 read their weights from
// the L2 three times.  With two exchanges of sums a row (mean, then squares) and scalar
// arithmetic: forward 5.8 to 6.6, backward 4.6 at 2048.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cpdr_internal.hpp"
#include "launch.cuh"
#include "norm_rows.cuh"
#include "vec_io.cuh"

namespace cpdr {
namespace {

using namespace vio;
using namespace norm;

// Each of the N values becomes its sum over the group of L lanes.
template <int L, int N>
__device__ __forceinline__ void lane_sums(float (&v)[N]) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Threads of a block: whole groups, 256 at least; 128 of three bf16 vectors, which
// leave one block of 256 an SM (the gradients of 2560 columns 4.5 -> 5.4 TB/s).
template <typename T, int TPR, int NV>
constexpr int kRowBlock = TPR >= 256 ? TPR : kVecOf<T> == 8 && NV == 3 ? (TPR < 128 ? 128 : TPR) : 256;

// What a warp's columns of a row come to: their mean `m + off`, the sum of
// squared differences to it, their share of the row; for the gradients the
// sums of u and of u times the differences.
struct Part {
    float m, off, sq, share, u, uc;
};
// Of a row: s - mean = (s - m) - shift, with the warp's own m.
struct Stats {
    float m, shift, sq, u, uc;
};

// Joins the warps' parts of R rows; `sh` holds R for each warp of the block, and
// may be written again once another barrier lies between.
template <int TPR, int R>
__device__ __forceinline__ void join(const Part (&own)[R], float n, Part (*sh)[R], Stats (&out)[R]) {
    if constexpr (TPR <= 32) {
#pragma unroll
        for (int r = 0; r < R; r++) out[r] = Stats{own[r].m, own[r].off, own[r].sq, own[r].u, own[r].uc};
    } else {
        constexpr int W = TPR / 32;
        const int w = threadIdx.x >> 5, w0 = w / W * W;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int r = 0; r < R; r++) sh[w][r] = own[r];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; r++) {
            const Part v = sh[w0 + (threadIdx.x & (W - 1))][r];   // every lane takes one warp's
            const float a = (v.m - own[r].m) + v.off;
            float one[2] = {v.share * a, v.u};
            lane_sums<W>(one);
            const float d = a - one[0];
            float two[2] = {fmaf(v.share * n * d, d, v.sq), fmaf(v.u, d, v.uc)};
            lane_sums<W>(two);
            out[r] = Stats{own[r].m, one[0], two[0], one[1], two[1]};
        }
    }
}

// Columns of this thread's warp (or of its row, where that is narrower) below `width`.
template <int TPR, int NV, int V>
__device__ __forceinline__ int warp_columns(int width) {
    constexpr int L = TPR < 32 ? TPR : 32;
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) n += max(0, min(L * V, width - (i * TPR + (int)(threadIdx.x % TPR) / L * L) * V));
    return n;
}

// The largest of R rows' values over the TPR threads of a row.
template <int TPR, int R>
__device__ __forceinline__ void row_max(float (&m)[R], float (*sh)[R]) {
    constexpr int LANES = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; r++) m[r] = max_nan(m[r], __shfl_xor_sync(0xffffffffu, m[r], o));
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int w = threadIdx.x >> 5, w0 = w / W * W;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int r = 0; r < R; r++) sh[w][r] = m[r];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; r++) {
            m[r] = sh[w0 + (threadIdx.x & (W - 1))][r];
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) m[r] = max_nan(m[r], __shfl_xor_sync(0xffffffffu, m[r], o));
        }
    }
}

// A 16-byte vector's values in pairs: H of them.
template <typename T>
constexpr int kPairs = kVecOf<T> / 2;
template <typename T, int H>
__device__ __forceinline__ void store_pairs(T *p, const float2 (&v)[H]) {
    float f[2 * H];
#pragma unroll
    for (int j = 0; j < H; j++) {
        f[2 * j] = v[j].x;
        f[2 * j + 1] = v[j].y;
    }
    store16(p, f);
}
template <int H>
__device__ __forceinline__ void load_pairs(const float *p, float2 (&v)[H]) {
#pragma unroll
    for (int j = 0; j < H; j += 2) {
        const float4 x = *reinterpret_cast<const float4 *>(p + 2 * j);
        v[j] = make_float2(x.x, x.y);
        v[j + 1] = make_float2(x.z, x.w);
    }
}

constexpr int kStages = 2;   // rows of a group of threads on their way to shared memory

struct FwdParams {
    const void *x, *res;
    const float *w, *b;
    void *s, *y;
    uint8_t *y8;
    float *scale;
    int64_t rows;
    int width;
    float eps, inv_width;
};

// Rows of a group of threads: without a residual two, as far as registers go.
template <int NV, bool RES>
constexpr int kFwdRows = NV > (RES ? 0 : 4) ? 1 : 2;

// Threads of a block, and blocks of an SM that the registers leave room for, by
// the vectors of a thread.
template <int TPR>
constexpr int kFwdBlock = TPR < 128 ? 128 : TPR;
constexpr int kFwdRegs[2][2][9] = {{{0, 48, 0, 104, 128}, {0, 40, 48, 64, 72, 0, 0, 0, 80}},
                                   {{0, 40, 56, 72, 88}, {0, 32, 40, 48, 56, 0, 0, 0, 96}}};
template <typename T, int TPR, int NV, bool RES>
constexpr int fwd_per_sm() {
    constexpr int regs = kFwdRegs[RES][kVecOf<T> == 4][NV];
    static_assert(regs > 0, "a form that no width runs");
    constexpr int n = 65536 / (regs * kFwdBlock<TPR>);
    return n < 1 ? 1 : n;
}

// grid: row blocks.  A group of threads takes one row, or without a residual two,
// whose loads take that one's place: both rows share the weights, and twice the
// bytes are in flight (TB/s with one row and with two: bf16 rows of 64 4.0 and 6.2, of
// 1360 4.9 and 5.5; fp32 of 128 4.0 and 6.7, of 776 5.9 and 6.7; of fp32 2048 6.9 both).
template <typename T, int TPR, int NV, bool E4M3, bool RES>
__global__ void __launch_bounds__(kFwdBlock<TPR>, fwd_per_sm<T, TPR, NV, RES>()) layernorm_fwd_kernel(FwdParams p) {
    constexpr int V = kVecOf<T>, H = kPairs<T>, W = kFwdBlock<TPR> / 32, L = TPR < 32 ? TPR : 32;
    constexpr int R = kFwdRows<NV, RES>, G = kFwdBlock<TPR> / TPR;
    __shared__ Part sh[W][R];
    __shared__ float sh_max[W][R];
    next_grid_may_start();
    previous_grid_done();
    const int64_t row0 = (int64_t)blockIdx.x * (G * R) + threadIdx.x / TPR;   // rows row0 + G r
    const int t = threadIdx.x % TPR;
    uint4 raw[RES ? 2 : 1][R][NV];   // x, and the residual
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int col = (i * TPR + t) * V;
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int64_t row = row0 + G * r, o = row * p.width + col;
            const bool live = row < p.rows && col < p.width;
            raw[0][r][i] = live ? load16((const T *)p.x + o) : make_uint4(0, 0, 0, 0);
            if (RES) raw[RES][r][i] = live ? load16((const T *)p.res + o) : make_uint4(0, 0, 0, 0);
        }
    }
    const float n_own = (float)warp_columns<TPR, NV, V>(p.width), inv_own = n_own > 0.f ? 1.f / n_own : 0.f;
    float2 s[R][NV][H];
    Part own[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int64_t row = row0 + G * r;
        float2 all = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            widen_pairs(raw[0][r][i], s[r][i]);
            if (RES) {
                float2 x[H];
                widen_pairs(raw[RES][r][i], x);
#pragma unroll
                for (int j = 0; j < H; j++) s[r][i][j] = add2(s[r][i][j], x[j]);
            }
            if (row < p.rows && col < p.width && p.s) store_pairs((T *)p.s + row * p.width + col, s[r][i]);
#pragma unroll
            for (int j = 0; j < H; j++) all = add2(all, s[r][i][j]);
        }
        float sum[1] = {all.x + all.y};
        lane_sums<L>(sum);
        const float m = sum[0] * inv_own;
        const float2 minus = both(-m);
        float2 diff = both(0.f), square = both(0.f);   // differences to the warp's mean, and their squares
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if ((i * TPR + t) * V < p.width) {
#pragma unroll
                for (int j = 0; j < H; j++) {
                    s[r][i][j] = add2(s[r][i][j], minus);
                    diff = add2(diff, s[r][i][j]);
                    square = fma2(s[r][i][j], s[r][i][j], square);
                }
            }
        }
        float st[2] = {diff.x + diff.y, square.x + square.y};
        lane_sums<L>(st);
        const float off = st[0] * inv_own;
        own[r] = Part{m, off, fmaf(-off, st[0], st[1]), n_own * p.inv_width, 0.f, 0.f};
    }
    Stats all[R];
    join<TPR, R>(own, (float)p.width, sh, all);
    float2 scale2[R], shift[R];
    float big[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const float rstd = rsqrtf(max_nan(all[r].sq * p.inv_width, 0.f) + p.eps);
        scale2[r] = both(rstd);
        shift[r] = both(-all[r].shift * rstd);
        big[r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int col = (i * TPR + t) * V;
        if (col >= p.width) continue;
        float2 w[H], b[H];
        load_pairs(p.w + col, w);
        if (p.b) load_pairs(p.b + col, b);
        else
#pragma unroll
            for (int j = 0; j < H; j++) b[j] = both(0.f);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int64_t row = row0 + G * r;
#pragma unroll
            for (int j = 0; j < H; j++) {
                s[r][i][j] = fma2(fma2(s[r][i][j], scale2[r], shift[r]), w[j], b[j]);
                if (E4M3) big[r] = max_nan(big[r], max_nan(fabsf(s[r][i][j].x), fabsf(s[r][i][j].y)));
            }
            if (row < p.rows && p.y) store_pairs((T *)p.y + row * p.width + col, s[r][i]);
        }
    }
    if (E4M3) {
        row_max<TPR, R>(big, sh_max);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int64_t row = row0 + G * r;
            if (row >= p.rows) continue;
            const float scale = max_nan(big[r] / kE4m3Max, 1.17549435e-38f);
            const float inv = 1.f / scale;
            if (t == 0) p.scale[row] = scale;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int col = (i * TPR + t) * V;
                float f[V];
#pragma unroll
                for (int j = 0; j < H; j++) {
                    f[2 * j] = s[r][i][j].x;
                    f[2 * j + 1] = s[r][i][j].y;
                }
                if (col < p.width) store_e4m3(p.y8 + row * p.width + col, f, inv);
            }
        }
    }
}

// bf16 rows of two vectors a thread, whose loads would wait too long for the
// exchanges between the warps: with the 8-bit output, whose largest value is
// a second exchange, and without a residual, where few bytes are in flight.
// The blocks are persistent, each group of threads takes every
// (gridDim.x * groups)-th row with the next ones on their way to shared memory,
// and the weights and biases stay in registers.  Rows of 4096: e4m3 with a residual 5.5 ->
// 6.5 TB/s, without one 5.0 -> 5.9.  Not for fp32, whose rows come from and go
// to too many places at once (5.6 TB/s instead of 7.0), nor for one vector (512
// columns to e4m3 5.7 instead of 6.7).
template <typename T, int NV>
constexpr bool kStream = kVecOf<T> == 8 && NV == 2;
template <typename T, int TPR, int NV>
constexpr int kept_per_sm() {
    constexpr int n = 65536 / (104 * kRowBlock<T, TPR, NV>);
    return n < 1 ? 1 : n;
}

template <typename T, int TPR, int NV, bool E4M3>
__global__ void __launch_bounds__(kRowBlock<T, TPR, NV>, kept_per_sm<T, TPR, NV>()) layernorm_stream_kernel(FwdParams p) {
    constexpr int V = kVecOf<T>, H = kPairs<T>, W = kRowBlock<T, TPR, NV> / 32, G = kRowBlock<T, TPR, NV> / TPR, L = TPR < 32 ? TPR : 32;
    constexpr int D = kStages;
    __shared__ Part sh[2][W][1];
    __shared__ float sh_max[W][1];
    extern __shared__ uint4 stage_sh[];   // [D][2 or 1][NV][threads]: x and the residual
    next_grid_may_start();
    previous_grid_done();
    const int t = threadIdx.x % TPR;
    const int64_t stride = (int64_t)gridDim.x * G;
    int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / TPR;
    const bool two = p.res != nullptr;
    auto place = [&](int stage, int which, int i) {
        return stage_sh + ((stage * (two ? 2 : 1) + which) * NV + i) * kRowBlock<T, TPR, NV> + threadIdx.x;
    };
    auto fetch = [&](int64_t at, int stage) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            const bool live = at < p.rows && col < p.width;
            const int64_t o = live ? at * p.width + col : 0;
            fetch16(place(stage, 0, i), (const T *)p.x + o, live);
            if (two) fetch16(place(stage, 1, i), (const T *)p.res + o, live);
        }
        fetch_group();
    };
#pragma unroll
    for (int d = 0; d < D; d++) fetch(row + d * stride, d);
    float2 w[NV][H], b[NV][H];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int col = (i * TPR + t) * V;
#pragma unroll
        for (int j = 0; j < H; j++) w[i][j] = b[i][j] = both(0.f);
        if (col < p.width) {
            load_pairs(p.w + col, w[i]);
            if (p.b) load_pairs(p.b + col, b[i]);
        }
    }
    const float n_own = (float)warp_columns<TPR, NV, V>(p.width), inv_own = n_own > 0.f ? 1.f / n_own : 0.f;
    int stage = 0, par = 0;
    // every group of the block makes the same number of turns (the barriers)
    for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += stride, row += stride) {
        const bool live = row < p.rows;
        const int64_t o = row * p.width;
        float2 s[NV][H];
        float2 all = both(0.f);
        fetch_wait<D - 1>();
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            widen_pairs(*place(stage, 0, i), s[i]);
            if (two) {
                float2 r[H];
                widen_pairs(*place(stage, 1, i), r);
#pragma unroll
                for (int j = 0; j < H; j++) s[i][j] = add2(s[i][j], r[j]);
            }
            if (live && col < p.width && p.s) store_pairs((T *)p.s + o + col, s[i]);
#pragma unroll
            for (int j = 0; j < H; j++) all = add2(all, s[i][j]);
        }
        fetch(row + D * stride, stage);
        stage = stage + 1 == D ? 0 : stage + 1;
        float sum[1] = {all.x + all.y};
        lane_sums<L>(sum);
        const float m = sum[0] * inv_own;
        const float2 minus = both(-m);
        float2 diff = both(0.f), square = both(0.f);   // differences to the warp's mean, and their squares
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if ((i * TPR + t) * V < p.width) {
#pragma unroll
                for (int j = 0; j < H; j++) {
                    s[i][j] = add2(s[i][j], minus);
                    diff = add2(diff, s[i][j]);
                    square = fma2(s[i][j], s[i][j], square);
                }
            }
        }
        float st[2] = {diff.x + diff.y, square.x + square.y};
        lane_sums<L>(st);
        const float off = st[0] * inv_own;
        const Part own[1] = {Part{m, off, fmaf(-off, st[0], st[1]), n_own * p.inv_width, 0.f, 0.f}};
        Stats joined[1];
        join<TPR, 1>(own, (float)p.width, sh[par], joined);
        par ^= 1;   // the next row's parts go to the other half: its barrier is behind these reads
        const float rstd = rsqrtf(max_nan(joined[0].sq * p.inv_width, 0.f) + p.eps);
        const float2 scale2 = both(rstd), shift = both(-joined[0].shift * rstd);
        float big[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
#pragma unroll
            for (int j = 0; j < H; j++) {
                s[i][j] = fma2(fma2(s[i][j], scale2, shift), w[i][j], b[i][j]);
                if (E4M3 && col < p.width) big[0] = max_nan(big[0], max_nan(fabsf(s[i][j].x), fabsf(s[i][j].y)));
            }
            if (live && col < p.width && p.y) store_pairs((T *)p.y + o + col, s[i]);
        }
        if (!E4M3) continue;
        row_max<TPR, 1>(big, sh_max);
        const float scale = max_nan(big[0] / kE4m3Max, 1.17549435e-38f);
        const float inv = 1.f / scale;
        if (live && t == 0) p.scale[row] = scale;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            float f[V];
#pragma unroll
            for (int j = 0; j < H; j++) {
                f[2 * j] = s[i][j].x;
                f[2 * j + 1] = s[i][j].y;
            }
            if (live && col < p.width) store_e4m3(p.y8 + o + col, f, inv);
        }
    }
    fetch_wait<0>();
}

struct BwdParams {
    const void *s, *dy, *dsum;
    const float *w;
    void *ds;
    float *part;         // [gridDim.x, 2 width]: dw, db
    int64_t rows;
    int width;
    float eps, inv_width;
};

constexpr int kBwdRegs[2][9] = {{0, 80, 128, 168, 128, 0, 0, 0, 0}, {0, 64, 96, 128, 128, 0, 0, 0, 128}};
template <typename T, int TPR, int NV>
constexpr int bwd_per_sm() {
    constexpr int n = 65536 / (kBwdRegs[kVecOf<T> == 4][NV] * kRowBlock<T, TPR, NV>);
    return n < 1 ? 1 : n;
}
// The weights, and later the block's sums, lie beside the stages where there
// is room for both (the widest fp32 rows have none).
template <typename T, int TPR, int NV>
constexpr int kBwdRowBytes = kRowBlock<T, TPR, NV> * NV * (kVecOf<T> * 4 + 48) <= 224 * 1024 ? kRowBlock<T, TPR, NV> * NV *kVecOf<T> * 4 : 0;
template <typename T, int TPR, int NV>
constexpr int bwd_stages() {
    constexpr int room = 200 * 1024 / bwd_per_sm<T, TPR, NV>() - kBwdRowBytes<T, TPR, NV>, stage = kRowBlock<T, TPR, NV> * NV * 48;
    constexpr int n = room / stage;
    return n < 1 ? 1 : n > kStages ? kStages : n;
}
// persistent: each group of TPR threads takes every (gridDim.x * groups)-th
// row and sums its rows' dw and db terms in registers; the block's sums go to its row of `part`.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(kRowBlock<T, TPR, NV>, bwd_per_sm<T, TPR, NV>()) layernorm_bwd_kernel(BwdParams p) {
    constexpr int V = kVecOf<T>, H = kPairs<T>, W = kRowBlock<T, TPR, NV> / 32;
    constexpr int G = kRowBlock<T, TPR, NV> / TPR, ROW = TPR * NV * V;
    constexpr int D = bwd_stages<T, TPR, NV>();
    constexpr int L = TPR < 32 ? TPR : 32;
    __shared__ Part sh[2][W][1];
    extern __shared__ __align__(16) float row_sh[];   // ROW weights, at the end the groups' sums; then the stages
    uint4 *stage_sh = reinterpret_cast<uint4 *>(row_sh + kBwdRowBytes<T, TPR, NV> / 4);   // [D][3][NV][threads]
    next_grid_may_start();
    previous_grid_done();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int64_t stride = (int64_t)gridDim.x * G;
    int64_t row = (int64_t)blockIdx.x * G + grp;
    auto place = [&](int stage, int which, int i) { return stage_sh + ((stage * 3 + which) * NV + i) * kRowBlock<T, TPR, NV> + threadIdx.x; };
    auto fetch = [&](int64_t at, int stage) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            const bool live = at < p.rows && col < p.width;
            const int64_t o = live ? at * p.width + col : 0;
            fetch16(place(stage, 0, i), (const T *)p.s + o, live);
            fetch16(place(stage, 1, i), (const T *)p.dy + o, live);
            if (p.dsum) fetch16(place(stage, 2, i), (const T *)p.dsum + o, live);
        }
        fetch_group();
    };
#pragma unroll
    for (int d = 0; d < D; d++) fetch(row + d * stride, d);
    constexpr bool NEAR = kBwdRowBytes<T, TPR, NV> > 0;
    static_assert(NEAR || G == 1, "the groups' sums need the room");
    if (NEAR)
        for (int i = threadIdx.x; i < ROW; i += kRowBlock<T, TPR, NV>) row_sh[i] = i < p.width ? p.w[i] : 0.f;
    auto weights = [&](int i, float2 (&w)[H]) {
        const int col = (i * TPR + t) * V;
        if (NEAR) {
            load_pairs(row_sh + col, w);
            return;
        }
#pragma unroll
        for (int j = 0; j < H; j++) w[j] = both(0.f);
        if (col < p.width) load_pairs(p.w + col, w);
    };
    int stage = 0, par = 0;
    const float n_own = (float)warp_columns<TPR, NV, V>(p.width), inv_own = n_own > 0.f ? 1.f / n_own : 0.f;
    float2 dw[NV][H], db[NV][H];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < H; j++) dw[i][j] = db[i][j] = both(0.f);
    __syncthreads();
    // every group of the block makes the same number of turns (the barriers)
    for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += stride, row += stride) {
        float2 s[NV][H], d[NV][H];
        float2 sum_s = both(0.f), sum_u = both(0.f);
        fetch_wait<D - 1>();
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float2 w[H];
            widen_pairs(*place(stage, 0, i), s[i]);
            widen_pairs(*place(stage, 1, i), d[i]);
            weights(i, w);
#pragma unroll
            for (int j = 0; j < H; j++) {
                sum_s = add2(sum_s, s[i][j]);
                sum_u = fma2(w[j], d[i][j], sum_u);
            }
        }
        float one[2] = {sum_s.x + sum_s.y, sum_u.x + sum_u.y};
        lane_sums<L>(one);
        const float m = one[0] * inv_own;
        const float2 minus_m = both(-m);
        float2 diff = both(0.f), square = both(0.f), prod = both(0.f);   // with c = s - m: sums of c, c^2 and u c
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if ((i * TPR + t) * V >= p.width) continue;
            float2 w[H];
            weights(i, w);
#pragma unroll
            for (int j = 0; j < H; j++) {
                s[i][j] = add2(s[i][j], minus_m);
                diff = add2(diff, s[i][j]);
                square = fma2(s[i][j], s[i][j], square);
                prod = fma2(mul2(w[j], d[i][j]), s[i][j], prod);
            }
        }
        float two[3] = {diff.x + diff.y, square.x + square.y, prod.x + prod.y};
        lane_sums<L>(two);
        const float off = two[0] * inv_own;
        const Part own[1] = {
            Part{m, off, fmaf(-off, two[0], two[1]), n_own * p.inv_width, one[1], fmaf(-off, one[1], two[2])}};
        Stats joined[1];
        join<TPR, 1>(own, (float)p.width, sh[par], joined);
        const Stats &all = joined[0];
        par ^= 1;   // the next row's parts go to the other half: its barrier is behind these reads
        // rows past the last are zeros: with eps of 0 their rstd would be infinite
        const float rstd = row < p.rows ? rsqrtf(max_nan(all.sq * p.inv_width, 0.f) + p.eps) : 0.f;
        const float mu = all.u * p.inv_width, dot = all.uc * p.inv_width * rstd;   // mean(u), mean(u xh)
        const float2 scale = both(rstd), shift = both(-all.shift * rstd), minus = both(-dot), minus_mu = both(-mu);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            float2 u[H], w[H];
            if (p.dsum) widen_pairs(*place(stage, 2, i), u);
            else
#pragma unroll
                for (int j = 0; j < H; j++) u[j] = both(0.f);
            weights(i, w);
#pragma unroll
            for (int j = 0; j < H; j++) {
                const float2 xh = fma2(s[i][j], scale, shift);
                dw[i][j] = fma2(d[i][j], xh, dw[i][j]);
                db[i][j] = add2(db[i][j], d[i][j]);
                u[j] = fma2(scale, fma2(xh, minus, fma2(w[j], d[i][j], minus_mu)), u[j]);
            }
            if (row < p.rows && col < p.width) store_pairs((T *)p.ds + row * p.width + col, u);
        }
        fetch(row + D * stride, stage);
        stage = stage + 1 == D ? 0 : stage + 1;
    }
    fetch_wait<0>();
    float *part = p.part + (int64_t)blockIdx.x * 2 * p.width;
#pragma unroll
    for (int which = 0; which < 2; which++) {
        auto value = [&](int i, int j) {
            const float2 v = which ? db[i][j / 2] : dw[i][j / 2];
            return j & 1 ? v.y : v.x;
        };
        if (G > 1) {
            __syncthreads();   // the weights, or the sums before, have been read
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < V; j++) row_sh[grp * ROW + (i * TPR + t) * V + j] = value(i, j);
            __syncthreads();
            for (int col = threadIdx.x; col < p.width; col += kRowBlock<T, TPR, NV>) {
                float v = 0.f;
                for (int i = 0; i < G; i++) v += row_sh[i * ROW + col];
                part[which * p.width + col] = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int col = (i * TPR + t) * V;
#pragma unroll
                for (int j = 0; j < V; j++)
                    if (col < p.width) part[which * p.width + col + j] = value(i, j);
            }
        }
    }
}

template <typename T, int TPR, int NV, bool RES>
int fwd_as(const FwdParams &p, void *st) {
    constexpr int per = kFwdBlock<TPR> / TPR * kFwdRows<NV, RES>;
    const int64_t grid = (p.rows + per - 1) / per;
    if (grid > (int64_t)0x7fffffff) return (int)cudaErrorInvalidValue;
    if constexpr (!kStream<T, NV>) {
        if (p.y8) return launch_early(layernorm_fwd_kernel<T, TPR, NV, true, RES>, dim3((unsigned)grid), kFwdBlock<TPR>, 0, 1, st, p);
    }
    return launch_early(layernorm_fwd_kernel<T, TPR, NV, false, RES>, dim3((unsigned)grid), kFwdBlock<TPR>, 0, 1, st, p);
}
template <typename T, int TPR, int NV>
int fwd(const FwdParams &p, int sms, void *st) {
    if constexpr (kStream<T, NV>) {
        constexpr int per = kRowBlock<T, TPR, NV> / TPR;
        if (p.y8 || !p.res)
            return launch_early(p.y8 ? layernorm_stream_kernel<T, TPR, NV, true> : layernorm_stream_kernel<T, TPR, NV, false>,
                                dim3((unsigned)std::min<int64_t>((p.rows + per - 1) / per, (int64_t)sms * kept_per_sm<T, TPR, NV>())),
                                kRowBlock<T, TPR, NV>, (size_t)kStages * (p.res ? 2 : 1) * NV * kRowBlock<T, TPR, NV> * 16, 1, st, p);
        return fwd_as<T, TPR, NV, true>(p, st);
    } else {
        return p.res ? fwd_as<T, TPR, NV, true>(p, st) : fwd_as<T, TPR, NV, false>(p, st);
    }
}

template <typename T, int TPR, int NV>
int bwd(const BwdParams &p, int grid, float *dw, float *db, void *st) {
    constexpr size_t smem = (size_t)kBwdRowBytes<T, TPR, NV> + (size_t)bwd_stages<T, TPR, NV>() * 3 * NV * kRowBlock<T, TPR, NV> * 16;
    static_assert(smem * bwd_per_sm<T, TPR, NV>() <= 224 * 1024, "the blocks of an SM fit its shared memory");
    const int rc = launch_early(layernorm_bwd_kernel<T, TPR, NV>, dim3((unsigned)grid), kRowBlock<T, TPR, NV>, smem, 1, st, p);
    if (rc) return rc;
    return launch_column_sums2(p.part, grid, p.width, dw, db, st);
}

// Threads and vectors of a row of the forward: as the RMS norm's, but 512 threads
// beyond 8192 bf16 columns.  They do not go by the outputs that are wanted: y
// has the same bits with and without y8.
template <typename T, typename F>
int by_width_fwd(int width, F f) {
    const int vecs = (width + kVecOf<T> - 1) / kVecOf<T>;
    if (vecs <= 768) return narrow_row<T>(vecs, f);
    if (vecs <= 1024) return with<256, 4>(f);
    if (vecs <= 1536) return with<512, 3>(f);
    if constexpr (kVecOf<T> == 4) {
        if (vecs > 2048) return with<512, 8>(f);
    }
    return with<512, 4>(f);
}
// Threads and vectors of a row of the backward, which holds dw and db: 512 threads
// beyond 768 vectors (of bf16 with two vectors where that does; one vector, half of the loads for each
// exchange between warps: rows of 1024 at 5.2 instead of 6.2 TB/s, of 4096 at 4.2 instead of 5.7).
template <typename T, typename F>
int by_width_bwd(int width, F f) {
    const int vecs = (width + kVecOf<T> - 1) / kVecOf<T>;
    if (vecs <= 768) return narrow_row<T>(vecs, f);
    if (vecs <= 1024) return with<512, 2>(f);
    if (vecs <= 1536) return with<512, 3>(f);
    if constexpr (kVecOf<T> == 4) {
        if (vecs > 2048) return with<512, 8>(f);
    }
    return with<512, 4>(f);
}

struct Shape {
    int rows, per_sm;   // rows of a block, blocks of an SM
};
template <typename T>
Shape bwd_shape(int width) {
    Shape s{};
    by_width_bwd<T>(width, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        s = Shape{kRowBlock<T, TPR, NV> / TPR, bwd_per_sm<T, TPR, NV>()};
        return CPDR_OK;
    });
    return s;
}

}  // namespace

static_assert(kMaxNormWidth <= 512 * 8 * kVecOf<float> && kMaxNormWidth <= 512 * 4 * kVecOf<__nv_bfloat16>, "a row fits the registers of one block");

int launch_layernorm_fwd(const cpdr_ctx *c, int64_t rows, int width, const void *x, const void *residual,
                         const float *weight, const float *bias, float eps, void *sum_out, void *y, void *y8,
                         float *scale, void *stream) {
    if (rows == 0) return 0;
    const FwdParams p{x, residual, weight, bias, sum_out, y, (uint8_t *)y8, scale, rows, width, eps, 1.f / (float)width};
    const int sms = device_sms(c->device);
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        return by_width_fwd<float>(width, [&](auto tpr, auto nv) {
            return fwd<float, decltype(tpr)::value, decltype(nv)::value>(p, sms, stream);
        });
    return by_width_fwd<__nv_bfloat16>(width, [&](auto tpr, auto nv) {
        return fwd<__nv_bfloat16, decltype(tpr)::value, decltype(nv)::value>(p, sms, stream);
    });
}

// Blocks of the backward: one wave, and no more than there are rows.
int layernorm_bwd_grid(const cpdr_ctx *c, int64_t rows, int width) {
    const Shape s = c->plan.in_dtype == CPDR_DTYPE_F32 ? bwd_shape<float>(width) : bwd_shape<__nv_bfloat16>(width);
    const int64_t blocks = (rows + s.rows - 1) / s.rows;
    return (int)std::max<int64_t>(1, std::min(blocks, (int64_t)device_sms(c->device) * s.per_sm));
}

int launch_layernorm_bwd(const cpdr_ctx *c, int64_t rows, int width, const void *s, const float *weight, float eps,
                         const void *dy, const void *dsum, void *ds, float *dweight, float *dbias, float *part,
                         void *stream) {
    const BwdParams p{s, dy, dsum, weight, ds, part, rows, width, eps, 1.f / (float)width};
    const int grid = layernorm_bwd_grid(c, rows, width);
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        return by_width_bwd<float>(width, [&](auto tpr, auto nv) {
            return bwd<float, decltype(tpr)::value, decltype(nv)::value>(p, grid, dweight, dbias, stream);
        });
    return by_width_bwd<__nv_bfloat16>(width, [&](auto tpr, auto nv) {
        return bwd<__nv_bfloat16, decltype(tpr)::value, decltype(nv)::value>(p, grid, dweight, dbias, stream);
    });
}

}  // namespace cpdr
