// RMS norm with the residual's addition, and its gradients.  Per row of
// `width` elements, with s = x + residual (or x),
//     rstd = 1 / sqrt(mean(s^2) + eps),   y_i = (s_i w_i) rstd,
// as T (fp32 or bf16), or as e4m3 with one scale per row,
//     scale = max(max_i |y_i| / 448, 2^-126),   y8_i = e4m3(y_i / scale);
// backward, from dy and (optionally) the gradient dsum that reaches s by the
// residual stream,
//     ds_i = rstd (w_i dy_i - s_i rstd^2 mean(s w dy)) + dsum_i,
//     dw_i = sum over rows of dy_i s_i rstd.
//
// Bound by HBM: every tensor is read and written once.  A row lives in the
// registers of one group of threads (1 to 1024 of them, one to four 16-byte
// vectors each), which needs one reduction for everything: the e4m3 row's
// largest |s w| comes with the sum of squares, since rounding is monotonic
// and rstd is one number per row, so max|y| is max|s w| times rstd exactly.
// Sums, statistics and dw are fp32; s is rounded once where it is stored, and
// y is computed from the unrounded sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cpdr_internal.hpp"
#include "launch.cuh"
#include "vec_io.cuh"

namespace cpdr {
namespace {

using namespace vio;

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

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

template <int TPR>
constexpr int kBlock = TPR < 256 ? 256 : TPR;

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

// grid: row blocks of kBlock / TPR rows
template <typename T, int TPR, int NV, bool E4M3>
__global__ void __launch_bounds__(kBlock<TPR>) rmsnorm_fwd_kernel(FwdParams p) {
    constexpr int V = kVecOf<T>;
    __shared__ float2 sh[64];
    next_grid_may_start();
    previous_grid_done();
    const int64_t row = (int64_t)blockIdx.x * (kBlock<TPR> / TPR) + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    const bool live = row < p.rows;
    const int64_t o = row * p.width;
    const T *x = (const T *)p.x + o;
    const T *res = p.res ? (const T *)p.res + o : nullptr;
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
        if (E4M3) {
            uint32_t q[V / 4];
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const uint32_t lo =
                    __nv_cvt_float2_to_fp8x2(make_float2(s[i][j] * inv, s[i][j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[i][j + 2] * inv, s[i][j + 3] * inv),
                                                             __NV_SATFINITE, __NV_E4M3);
                q[j / 4] = lo | hi << 16;
            }
            uint8_t *d = p.y8 + o + col;
            if (V == 8)
                *reinterpret_cast<uint2 *>(d) = make_uint2(q[0], q[V / 4 - 1]);
            else
                *reinterpret_cast<uint32_t *>(d) = q[0];
        }
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

// persistent: each group of TPR threads takes every (gridDim.x * groups)-th
// row, with the next row's loads in flight, and sums its rows' dw terms in
// registers; the block's sum goes to its row of `part`.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(kBlock<TPR>) rmsnorm_bwd_kernel(BwdParams p) {
    constexpr int V = kVecOf<T>;
    constexpr int G = kBlock<TPR> / TPR;
    __shared__ float2 sh[64];
    extern __shared__ float dw_sh[];
    next_grid_may_start();
    previous_grid_done();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int64_t stride = (int64_t)gridDim.x * G;
    const T *sp = (const T *)p.s, *dyp = (const T *)p.dy, *dsp = (const T *)p.dsum;
    float w[NV][V], dw[NV][V];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int col = (i * TPR + t) * V;
#pragma unroll
        for (int j = 0; j < V; j++) {
            w[i][j] = col < p.width ? p.w[col + j] : 0.f;
            dw[i][j] = 0.f;
        }
    }
    uint4 sr[NV], dr[NV], ur[NV];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            sr[i] = dr[i] = ur[i] = make_uint4(0, 0, 0, 0);
            if (row < p.rows && col < p.width) {
                const int64_t o = row * p.width + col;
                sr[i] = load16(sp + o);
                dr[i] = load16(dyp + o);
                if (dsp) ur[i] = load16(dsp + o);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * G + grp;
    load(row);
    int par = 0;
    // every group of the block makes the same number of turns (the barriers)
    for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += stride, row += stride, par ^= 1) {
        float s[NV][V], d[NV][V], u[NV][V];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            widen16(sr[i], s[i]);
            widen16(dr[i], d[i]);
            widen16(ur[i], u[i]);
        }
        load(row + stride);
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < V; j++) {
                ss = fmaf(s[i][j], s[i][j], ss);
                dot = fmaf(s[i][j], w[i][j] * d[i][j], dot);
            }
        const float2 st = row_reduce<TPR, false>(ss, dot, sh, par);
        const float rstd = rsqrtf(fmaf(st.x, p.inv_width, p.eps));
        const float k = rstd * rstd * (st.y * p.inv_width);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            float ds[V];
#pragma unroll
            for (int j = 0; j < V; j++) {
                dw[i][j] = fmaf(d[i][j], s[i][j] * rstd, dw[i][j]);
                ds[j] = fmaf(rstd, fmaf(w[i][j], d[i][j], -k * s[i][j]), u[i][j]);
            }
            if (row < p.rows && col < p.width) store16((T *)p.ds + row * p.width + col, ds);
        }
    }
    float *part = p.part + (int64_t)blockIdx.x * p.width;
    if (G > 1) {
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < V; j++) dw_sh[grp * (TPR * NV * V) + (i * TPR + t) * V + j] = dw[i][j];
        __syncthreads();
        for (int col = threadIdx.x; col < p.width; col += kBlock<TPR>) {
            float v = 0.f;
            for (int i = 0; i < G; i++) v += dw_sh[i * (TPR * NV * V) + col];
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
// column, then those 16.
__global__ void __launch_bounds__(kSumCols *kSumRows)
column_sums_kernel(const float *__restrict__ part, int nparts, int width, float *__restrict__ out) {
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
        out[col] = v;
    }
}

template <typename T, int TPR, int NV>
int fwd(const FwdParams &p, cudaStream_t st) {
    constexpr int per = kBlock<TPR> / TPR;
    const int64_t grid = (p.rows + per - 1) / per;
    if (grid > (int64_t)0x7fffffff) return (int)cudaErrorInvalidValue;
    return launch_early(p.y8 ? rmsnorm_fwd_kernel<T, TPR, NV, true> : rmsnorm_fwd_kernel<T, TPR, NV, false>,
                        dim3((unsigned)grid), kBlock<TPR>, 0, 1, st, p);
}

template <typename T, int TPR, int NV>
int bwd(const BwdParams &p, int grid, float *dw, cudaStream_t st) {
    constexpr int G = kBlock<TPR> / TPR;
    const size_t smem = G > 1 ? (size_t)G * TPR * NV * kVecOf<T> * sizeof(float) : 0;
    static_assert((G > 1 ? G * TPR * NV * kVecOf<T> * 4 : 0) <= 48 * 1024, "dw staging within the default shared memory");
    const int rc = launch_early(rmsnorm_bwd_kernel<T, TPR, NV>, dim3((unsigned)grid), kBlock<TPR>, smem, 1, st, p);
    if (rc) return rc;
    return launch_column_sums(p.part, grid, p.width, dw, st);
}

// Threads per row: one 16-byte vector each for rows of up to 32 vectors, two
// for wider ones, four for the widest fp32 rows.
template <typename T, typename F>
int by_width(int width, F f) {
    const int vecs = (width + kVecOf<T> - 1) / kVecOf<T>;
    if (vecs <= 1) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 1>());
    if (vecs <= 2) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 1>());
    if (vecs <= 4) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    if (vecs <= 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    if (vecs <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (vecs <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
    if (vecs <= 64) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
    if (vecs <= 128) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    if (vecs <= 256) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
    if (vecs <= 512) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
    if (vecs <= 1024) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
    if constexpr (kVecOf<T> == 4) {
        if (vecs > 2048) return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
    }
    return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
}

int rows_per_block(int width, bool f32) {
    auto g = [](auto tpr, auto) { return kBlock<decltype(tpr)::value> / decltype(tpr)::value; };
    return f32 ? by_width<float>(width, g) : by_width<__nv_bfloat16>(width, g);
}

}  // namespace

static_assert(kMaxNormWidth <= 1024 * 4 * kVecOf<float> && kMaxNormWidth <= 1024 * 2 * kVecOf<__nv_bfloat16>, "a row fits the registers of one block");

int launch_column_sums(const float *part, int nparts, int width, float *out, void *stream) {
    return launch_early(column_sums_kernel, dim3((unsigned)((width + kSumCols - 1) / kSumCols)), kSumCols * kSumRows, 0, 1, stream,
                        part, nparts, width, out);
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

// Blocks of the backward: four per SM (one for rows of 1024 threads), and no
// more than there are rows.
int rmsnorm_bwd_grid(const cpdr_ctx *c, int64_t rows, int width) {
    const int per = rows_per_block(width, c->plan.in_dtype == CPDR_DTYPE_F32);
    const int64_t blocks = (rows + per - 1) / per;
    const int64_t most = (int64_t)device_sms(c->device) * (width > 4096 ? 2 : 4);
    return (int)std::max<int64_t>(1, std::min(blocks, most));
}

int launch_rmsnorm_bwd(const cpdr_ctx *c, int64_t rows, int width, const void *s, const float *weight, float eps,
                       const void *dy, const void *dsum, void *ds, float *dweight, float *part, void *stream) {
    BwdParams p{s, dy, dsum, weight, ds, part, rows, width, eps, 1.f / (float)width};
    const int grid = rmsnorm_bwd_grid(c, rows, width);
    cudaStream_t st = (cudaStream_t)stream;
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        return by_width<float>(width, [&](auto tpr, auto nv) {
            return bwd<float, decltype(tpr)::value, decltype(nv)::value>(p, grid, dweight, st);
        });
    return by_width<__nv_bfloat16>(width, [&](auto tpr, auto nv) {
        return bwd<__nv_bfloat16, decltype(tpr)::value, decltype(nv)::value>(p, grid, dweight, st);
    });
}

}  // namespace cpdr
