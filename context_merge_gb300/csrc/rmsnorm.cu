// RMS norm with the residual's addition, and its gradients.  Per row of
// `width` elements, with s = x + residual (or x),
//     rstd = 1 / sqrt(mean(s^2) + eps),   y_i = (s_i w_i) rstd,
// as T (fp32 or bf16), or as e4m3 with one scale per row,
//     scale = max(max_i |y_i| / 448, 2^-126),   y8_i = e4m3(y_i (1 / scale));
// backward, from dy and (optionally) the gradient dsum that reaches s by the
// residual stream,
//     ds_i = rstd (w_i dy_i - s_i rstd^2 mean(s w dy)) + dsum_i,
//     dw_i = sum over rows of dy_i s_i rstd.
//
// Bound by HBM: every tensor is read and written once.  A row lives in the
// registers of one group of threads (1 to 512 of them, one to eight 16-byte
// vectors each), which needs one reduction for everything: the e4m3 row's
// largest |s w| comes with the sum of squares, since rounding is monotonic
// and rstd is one number per row, so max|y| is max|s w| times rstd exactly.
// Sums, statistics and dw are fp32; s is rounded once where it is stored, and
// y is computed from the unrounded sum.
//
// Measured over 0.4 GB a tensor: forward 6.8 to 7.1 TB/s (bf16 with a
// residual, 72 to 12288 columns; 6.1 at 16384) and 6.4 to 7.1 (fp32); backward
// 4.9 to 6.1 TB/s up to 2048 columns of bf16, 4.1 to 5.3 up to 8192 and 3.8 to
// 4.5 beyond, and of fp32 5.9 to 6.7 up to 6144 columns and 4.6 to 5.6 beyond:
// few wide rows are in flight in an SM.
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

// Sum of `s` and combination of `m` (maximum, or sum) over the TPR threads
// of a row; `sh` holds a pair per warp of the block, one half for each parity.
template <int TPR, bool MAX>
__device__ __forceinline__ float2 row_reduce(float s, float m, float2 *sh, int par) {
    constexpr int LANES = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        const float t = __shfl_xor_sync(0xffffffffu, m, o);
        m = MAX ? max_nan(m, t) : m + t;
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float2 *mine = sh + par * 32;
        const int w = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) mine[w] = make_float2(s, m);
        __syncthreads();
        const int w0 = w / W * W;
        float2 v = mine[w0];
        s = v.x;
        m = v.y;
#pragma unroll
        for (int i = 1; i < W; i++) {
            v = mine[w0 + i];
            s += v.x;
            m = MAX ? max_nan(m, v.y) : m + v.y;
        }
    }
    return make_float2(s, m);
}

struct FwdParams {
    const void *x, *res;
    const float *w;
    void *s, *y;
    uint8_t *y8;
    float *scale;
    int64_t rows;
    int width;
    float eps, inv_width;
};

// Wide fp32 rows without a residual have few loads in flight: they take 64
// registers a thread, 1024 threads an SM (16384 columns 4.5 -> 6.9 TB/s; with
// a residual that costs spills, 6.9 -> 5.9).
template <typename T, int NV, bool RES>
constexpr bool kFwdSlim = kVecOf<T> == 4 && NV >= 4 && !RES;

// grid: row blocks of kBlock / TPR rows; RES: a residual may be given
template <typename T, int TPR, int NV, bool E4M3, bool RES>
__global__ void __launch_bounds__(kBlock<TPR>, kFwdSlim<T, NV, RES> ? 1024 / TPR : 1) rmsnorm_fwd_kernel(FwdParams p) {
    constexpr int V = kVecOf<T>;
    __shared__ float2 sh[64];
    next_grid_may_start();
    previous_grid_done();
    const int64_t row = (int64_t)blockIdx.x * (kBlock<TPR> / TPR) + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    const bool live = row < p.rows;
    const int64_t o = row * p.width;
    const T *x = (const T *)p.x + o;
    const T *res = RES && p.res ? (const T *)p.res + o : nullptr;
    uint4 xr[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int col = (i * TPR + t) * V;
        xr[i] = rr[i] = make_uint4(0, 0, 0, 0);
        if (live && col < p.width) {
            xr[i] = load16(x + col);
            if (res) rr[i] = load16(res + col);
        }
    }
    float s[NV][V];
    float sum = 0.f, big = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int col = (i * TPR + t) * V;
        float r[V];
        widen16(xr[i], s[i]);
        if (res) {
            widen16(rr[i], r);
#pragma unroll
            for (int j = 0; j < V; j++) s[i][j] += r[j];
        }
        if (live && col < p.width && p.s) store16((T *)p.s + o + col, s[i]);
#pragma unroll
        for (int j = 0; j < V; j++) sum = fmaf(s[i][j], s[i][j], sum);
        // from here on s is s w
        if (col < p.width) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(p.w + col + j);
                s[i][j] *= w.x;
                s[i][j + 1] *= w.y;
                s[i][j + 2] *= w.z;
                s[i][j + 3] *= w.w;
            }
            if (E4M3) {
#pragma unroll
                for (int j = 0; j < V; j++) big = max_nan(big, fabsf(s[i][j]));
            }
        }
    }
    const float2 st = row_reduce<TPR, true>(sum, big, sh, 0);
    const float rstd = rsqrtf(fmaf(st.x, p.inv_width, p.eps));
    if (!live) return;
    float inv = 0.f;
    if (E4M3) {
        const float scale = max_nan(st.y * rstd / kE4m3Max, 1.17549435e-38f);
        inv = 1.f / scale;
        if (t == 0) p.scale[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int col = (i * TPR + t) * V;
        if (col >= p.width) continue;
#pragma unroll
        for (int j = 0; j < V; j++) s[i][j] *= rstd;
        if (p.y) store16((T *)p.y + o + col, s[i]);
        if (E4M3) store_e4m3(p.y8 + o + col, s[i], inv);
    }
}

struct BwdParams {
    const void *s, *dy, *dsum;
    const float *w;
    void *ds;
    float *part;         // [gridDim.x, width]
    int64_t rows;
    int width;
    float eps, inv_width;
};

// Blocks of an SM that the backward's registers leave room for: its grid, one
// wave of them, and the bound that holds the compiler to it.  Spills cost more
// than the missing warps: rows of 12288 ran at 1.6 TB/s as 1024 threads of 64
// registers, at 4.3 (bf16) and 5.3 (fp32) as 512 of 128.
template <typename T, int TPR, int NV>
constexpr int bwd_per_sm() {
    constexpr bool f32 = kVecOf<T> == 4;
    if (kBlock<TPR> > 256) return 1;
    if (NV == 1) return f32 ? 6 : 5;
    if (!f32 || NV > 3) return 2;
    return NV == 2 ? 4 : 3;
}
// More blocks do more than the next row's loads in flight (128 columns 5.2 ->
// 6.0 TB/s in bf16, fp32 rows of 4096 4.2 -> 6.1), but for two bf16 vectors,
// whose 32 sums and products leave two blocks an SM (8192 columns 5.3 TB/s
// with the loads ahead, 3.7 without).
template <typename T, int NV>
constexpr bool kBwdAhead = NV == 2 && kVecOf<T> == 8;

// persistent: each group of TPR threads takes every (gridDim.x * groups)-th
// row and sums its rows' dw terms in registers; the block's sum goes to its row of `part`.  The weights lie in
// shared memory and the row stays as it was loaded (widened where it is used,
// twice), so that registers are left for the loads in flight.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(kBlock<TPR>, bwd_per_sm<T, TPR, NV>()) rmsnorm_bwd_kernel(BwdParams p) {
    constexpr int V = kVecOf<T>;
    constexpr int G = kBlock<TPR> / TPR, ROW = TPR * NV * V;
    constexpr bool AHEAD = kBwdAhead<T, NV>;
    __shared__ float2 sh[64];
    extern __shared__ __align__(16) float row_sh[];   // ROW weights; at the end the groups' dw
    next_grid_may_start();
    previous_grid_done();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int64_t stride = (int64_t)gridDim.x * G;
    const T *sp = (const T *)p.s, *dyp = (const T *)p.dy, *dsp = (const T *)p.dsum;
    for (int i = threadIdx.x; i < ROW; i += kBlock<TPR>) row_sh[i] = i < p.width ? p.w[i] : 0.f;
    float dw[NV][V];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < V; j++) dw[i][j] = 0.f;
    struct Raw {
        uint4 s[NV], d[NV], u[NV];
    };
    auto load = [&](Raw &r, int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            r.s[i] = r.d[i] = r.u[i] = make_uint4(0, 0, 0, 0);
            if (row < p.rows && col < p.width) {
                const int64_t o = row * p.width + col;
                r.s[i] = load16(sp + o);
                r.d[i] = load16(dyp + o);
                if (dsp) r.u[i] = load16(dsp + o);
            }
        }
    };
    auto weights = [&](int i, float (&w)[V]) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(row_sh + (i * TPR + t) * V + j);
            w[j] = v.x;
            w[j + 1] = v.y;
            w[j + 2] = v.z;
            w[j + 3] = v.w;
        }
    };
    __syncthreads();
    int64_t row = (int64_t)blockIdx.x * G + grp;
    Raw cur, next;
    if (AHEAD) load(cur, row);
    int par = 0;
    // every group of the block makes the same number of turns (the barriers)
    for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += stride, row += stride, par ^= 1) {
        if (AHEAD) load(next, row + stride);
        else load(cur, row);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float s[V], d[V], w[V];
            widen16(cur.s[i], s);
            widen16(cur.d[i], d);
            weights(i, w);
#pragma unroll
            for (int j = 0; j < V; j++) {
                ss = fmaf(s[j], s[j], ss);
                dot = fmaf(s[j], w[j] * d[j], dot);
            }
        }
        const float2 st = row_reduce<TPR, false>(ss, dot, sh, par);
        // rows past the last are zeros: with eps of 0 their rstd would be infinite
        const float rstd = row < p.rows ? rsqrtf(fmaf(st.x, p.inv_width, p.eps)) : 0.f;
        const float k = rstd * rstd * (st.y * p.inv_width);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            float s[V], d[V], u[V], w[V], ds[V];
            widen16(cur.s[i], s);
            widen16(cur.d[i], d);
            widen16(cur.u[i], u);
            weights(i, w);
#pragma unroll
            for (int j = 0; j < V; j++) {
                dw[i][j] = fmaf(d[j], s[j] * rstd, dw[i][j]);
                ds[j] = fmaf(rstd, fmaf(w[j], d[j], -k * s[j]), u[j]);
            }
            if (row < p.rows && col < p.width) store16((T *)p.ds + row * p.width + col, ds);
        }
        if (AHEAD) cur = next;
    }
    float *part = p.part + (int64_t)blockIdx.x * p.width;
    if (G > 1) {
        __syncthreads();   // the weights have been read
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < V; j++) row_sh[grp * ROW + (i * TPR + t) * V + j] = dw[i][j];
        __syncthreads();
        for (int col = threadIdx.x; col < p.width; col += kBlock<TPR>) {
            float v = 0.f;
            for (int i = 0; i < G; i++) v += row_sh[i * ROW + col];
            part[col] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
#pragma unroll
            for (int j = 0; j < V; j++)
                if (col < p.width) part[col + j] = dw[i][j];
        }
    }
}

constexpr int kSumCols = 32, kSumRows = 16;

// out[col] = sum of part[:, col], in a fixed order: 16 strided sums per
// column, then those 16.  Columns from `split` on go to out2 (NULL: nowhere).
__global__ void __launch_bounds__(kSumCols *kSumRows)
column_sums_kernel(const float *part, int nparts, int width, float *out, int split, float *out2) {
    __shared__ float sh[kSumRows][kSumCols + 1];
    next_grid_may_start();
    previous_grid_done();
    const int cx = threadIdx.x % kSumCols, ry = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + cx;
    float v = 0.f;
    if (col < width)
        for (int r = ry; r < nparts; r += kSumRows) v += part[(int64_t)r * width + col];
    sh[ry][cx] = v;
    __syncthreads();
    if (ry == 0 && col < width) {
        v = sh[0][cx];
#pragma unroll
        for (int r = 1; r < kSumRows; r++) v += sh[r][cx];
        if (col < split) out[col] = v;
        else if (out2) out2[col - split] = v;
    }
}

template <typename T, int TPR, int NV, bool RES>
int fwd_as(const FwdParams &p, cudaStream_t st) {
    constexpr int per = kBlock<TPR> / TPR;
    const int64_t grid = (p.rows + per - 1) / per;
    if (grid > (int64_t)0x7fffffff) return (int)cudaErrorInvalidValue;
    return launch_early(p.y8 ? rmsnorm_fwd_kernel<T, TPR, NV, true, RES> : rmsnorm_fwd_kernel<T, TPR, NV, false, RES>,
                        dim3((unsigned)grid), kBlock<TPR>, 0, 1, st, p);
}
template <typename T, int TPR, int NV>
int fwd(const FwdParams &p, cudaStream_t st) {
    if constexpr (kFwdSlim<T, NV, false>) {
        if (!p.res) return fwd_as<T, TPR, NV, false>(p, st);
    }
    return fwd_as<T, TPR, NV, true>(p, st);
}

template <typename T, int TPR, int NV>
int bwd(const BwdParams &p, int grid, float *dw, cudaStream_t st) {
    constexpr int G = kBlock<TPR> / TPR;
    constexpr size_t smem = (size_t)G * TPR * NV * kVecOf<T> * sizeof(float);
    static_assert(smem * bwd_per_sm<T, TPR, NV>() <= 220 * 1024, "the blocks of an SM fit its shared memory");
    const int rc = launch_early(rmsnorm_bwd_kernel<T, TPR, NV>, dim3((unsigned)grid), kBlock<TPR>, smem, 1, st, p);
    if (rc) return rc;
    return launch_column_sums(p.part, grid, p.width, dw, st);
}

// Threads and vectors of a row: as narrow_row, and up to eight vectors for wide rows.
template <typename T, typename F>
int by_width(int width, F f) {
    const int vecs = (width + kVecOf<T> - 1) / kVecOf<T>;
    if (vecs <= 768) return narrow_row<T>(vecs, f);
    if (vecs <= 1024) return with<256, 4>(f);
    if (vecs <= 1536) return with<256, 6>(f);
    if constexpr (kVecOf<T> == 4) {
        if (vecs > 2048) return with<512, 8>(f);
    }
    return with<256, 8>(f);
}
// The same for the backward, whose thread holds dw besides: 512 threads a row
// where the eight values of a bf16 vector, or eight vectors, would take too
// many registers (fp32 rows of 6144 run at 6.6 TB/s as 256 x 6, at 4.9 as
// 512 x 3; bf16 rows of 12288 at 4.0 and 4.3), and one bf16 vector instead of
// two up to 128 threads (1024 columns 4.5 -> 5.3).
template <typename T, typename F>
int by_width_bwd(int width, F f) {
    const int vecs = (width + kVecOf<T> - 1) / kVecOf<T>;
    if constexpr (kVecOf<T> == 8) {
        if (vecs > 48 && vecs <= 64) return with<64, 1>(f);
        if (vecs > 96 && vecs <= 128) return with<128, 1>(f);
    }
    if (vecs <= 768) return narrow_row<T>(vecs, f);
    if constexpr (kVecOf<T> == 4) {
        if (vecs <= 1024) return with<256, 4>(f);
        if (vecs <= 1536) return with<256, 6>(f);
        if (vecs > 2048) return with<512, 8>(f);
    } else {
        if (vecs <= 1024) return with<512, 2>(f);
        if (vecs <= 1536) return with<512, 3>(f);
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
        constexpr int TPR = decltype(tpr)::value;
        s = Shape{kBlock<TPR> / TPR, bwd_per_sm<T, TPR, decltype(nv)::value>()};
        return CPDR_OK;
    });
    return s;
}

}  // namespace

static_assert(kMaxNormWidth <= 512 * 8 * kVecOf<float> && kMaxNormWidth <= 512 * 4 * kVecOf<__nv_bfloat16>, "a row fits the registers of one block");

int launch_column_sums(const float *part, int nparts, int width, float *out, void *stream) {
    return launch_early(column_sums_kernel, dim3((unsigned)((width + kSumCols - 1) / kSumCols)), kSumCols * kSumRows, 0, 1, stream,
                        part, nparts, width, out, width, (float *)nullptr);
}

int launch_column_sums2(const float *part, int nparts, int width, float *out, float *out2, void *stream) {
    return launch_early(column_sums_kernel, dim3((unsigned)((2 * width + kSumCols - 1) / kSumCols)), kSumCols * kSumRows, 0, 1,
                        stream, part, nparts, 2 * width, out, width, out2);
}

int launch_rmsnorm_fwd(const cpdr_ctx *c, int64_t rows, int width, const void *x, const void *residual,
                       const float *weight, float eps, void *sum_out, void *y, void *y8, float *scale, void *stream) {
    if (rows == 0) return 0;
    FwdParams p{x, residual, weight, sum_out, y, (uint8_t *)y8, scale, rows, width, eps, 1.f / (float)width};
    cudaStream_t st = (cudaStream_t)stream;
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        return by_width<float>(width, [&](auto tpr, auto nv) {
            return fwd<float, decltype(tpr)::value, decltype(nv)::value>(p, st);
        });
    return by_width<__nv_bfloat16>(width, [&](auto tpr, auto nv) {
        return fwd<__nv_bfloat16, decltype(tpr)::value, decltype(nv)::value>(p, st);
    });
}

// Blocks of the backward: one wave, and no more than there are rows.
int rmsnorm_bwd_grid(const cpdr_ctx *c, int64_t rows, int width) {
    const Shape s = c->plan.in_dtype == CPDR_DTYPE_F32 ? bwd_shape<float>(width) : bwd_shape<__nv_bfloat16>(width);
    const int64_t blocks = (rows + s.rows - 1) / s.rows;
    return (int)std::max<int64_t>(1, std::min(blocks, (int64_t)device_sms(c->device) * s.per_sm));
}

int launch_rmsnorm_bwd(const cpdr_ctx *c, int64_t rows, int width, const void *s, const float *weight, float eps,
                       const void *dy, const void *dsum, void *ds, float *dweight, float *part, void *stream) {
    BwdParams p{s, dy, dsum, weight, ds, part, rows, width, eps, 1.f / (float)width};
    const int grid = rmsnorm_bwd_grid(c, rows, width);
    cudaStream_t st = (cudaStream_t)stream;
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        return by_width_bwd<float>(width, [&](auto tpr, auto nv) {
            return bwd<float, decltype(tpr)::value, decltype(nv)::value>(p, grid, dweight, st);
        });
    return by_width_bwd<__nv_bfloat16>(width, [&](auto tpr, auto nv) {
        return bwd<__nv_bfloat16, decltype(tpr)::value, decltype(nv)::value>(p, grid, dweight, st);
    });
}

}  // namespace cpdr
