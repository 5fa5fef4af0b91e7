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
// to the mean, which a row with a large mean needs.  The fp32 mean is itself off by
// some half steps of the row's size; the sum of the differences, which comes
// with their squares, says by how much, and both are corrected by it.
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

// Each of the N values becomes its sum over the TPR threads of a row.  `sh`
// holds N floats per warp; a second call may take the same place once another
// one, which has a barrier, lies between.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*sh)[N]) {
    constexpr int LANES = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int w = threadIdx.x >> 5, w0 = w / W * W;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; i++) sh[w][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = sh[w0][i];
#pragma unroll
        for (int x = 1; x < W; x++)
#pragma unroll
            for (int i = 0; i < N; i++) v[i] += sh[w0 + x][i];
    }
}

template <int TPR>
__device__ __forceinline__ float row_max(float m, float *sh) {
    constexpr int LANES = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int w = threadIdx.x >> 5, w0 = w / W * W;
        if ((threadIdx.x & 31) == 0) sh[w] = m;
        __syncthreads();
        m = sh[w0];
#pragma unroll
        for (int x = 1; x < W; x++) m = max_nan(m, sh[w0 + x]);
    }
    return m;
}

template <int V>
__device__ __forceinline__ void load_floats(const float *p, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p + j);
        v[j] = x.x;
        v[j + 1] = x.y;
        v[j + 2] = x.z;
        v[j + 3] = x.w;
    }
}

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

// Blocks of an SM that the forward's registers leave room for.
template <typename T, int TPR, int NV>
constexpr int fwd_per_sm() {
    constexpr int regs = kVecOf<T> == 8 ? (NV == 1 ? 48 : NV == 2 ? 64 : NV == 3 ? 80 : 128)
                                        : (NV <= 2 ? 48 : NV == 3 ? 56 : NV == 4 ? 64 : 128);
    constexpr int n = 65536 / (regs * kBlock<TPR>);
    return n < 1 ? 1 : n;
}

// persistent: each group of TPR threads takes every (gridDim.x * groups)-th row,
// whose loads go out before the reductions of the row before it.
template <typename T, int TPR, int NV, bool E4M3>
__global__ void __launch_bounds__(kBlock<TPR>, fwd_per_sm<T, TPR, NV>()) layernorm_fwd_kernel(FwdParams p) {
    constexpr int V = kVecOf<T>, W = kBlock<TPR> / 32, G = kBlock<TPR> / TPR;
    __shared__ float sh1[W][1], sh2[W][2], sh3[W];
    next_grid_may_start();
    previous_grid_done();
    const int t = threadIdx.x % TPR;
    const int64_t stride = (int64_t)gridDim.x * G;
    int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / TPR;
    uint4 xr[NV], rr[NV];
    auto load = [&](int64_t at) {
        const T *x = (const T *)p.x + at * p.width, *res = p.res ? (const T *)p.res + at * p.width : nullptr;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            xr[i] = rr[i] = make_uint4(0, 0, 0, 0);
            if (at < p.rows && col < p.width) {
                xr[i] = load16(x + col);
                if (res) rr[i] = load16(res + col);
            }
        }
    };
    load(row);
    // every group of the block makes the same number of turns (the barriers)
    for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += stride, row += stride) {
        const bool live = row < p.rows;
        const int64_t o = row * p.width;
        float s[NV][V];
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            widen16(xr[i], s[i]);
            if (p.res) {
                float r[V];
                widen16(rr[i], r);
#pragma unroll
                for (int j = 0; j < V; j++) s[i][j] += r[j];
            }
            if (live && col < p.width && p.s) store16((T *)p.s + o + col, s[i]);
#pragma unroll
            for (int j = 0; j < V; j++) sum[0] += s[i][j];
        }
        load(row + stride);
        row_sums<TPR>(sum, sh1);
        const float mean = sum[0] * p.inv_width;
        float st[2] = {0.f, 0.f};   // differences to the mean, and their squares
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if ((i * TPR + t) * V < p.width) {
#pragma unroll
                for (int j = 0; j < V; j++) {
                    s[i][j] -= mean;
                    st[0] += s[i][j];
                    st[1] = fmaf(s[i][j], s[i][j], st[1]);
                }
            }
        }
        row_sums<TPR>(st, sh2);
        const float off = st[0] * p.inv_width;
        const float rstd = rsqrtf(max_nan(fmaf(-off, off, st[1] * p.inv_width), 0.f) + p.eps);
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            if (col >= p.width) continue;
            float w[V], b[V];
            load_floats(p.w + col, w);
#pragma unroll
            for (int j = 0; j < V; j++) b[j] = 0.f;
            if (p.b) load_floats(p.b + col, b);
#pragma unroll
            for (int j = 0; j < V; j++) {
                s[i][j] = fmaf((s[i][j] - off) * rstd, w[j], b[j]);
                if (E4M3) big = max_nan(big, fabsf(s[i][j]));
            }
            if (live && p.y) store16((T *)p.y + o + col, s[i]);
        }
        if (E4M3) {
            const float scale = max_nan(row_max<TPR>(big, sh3) / kE4m3Max, 1.17549435e-38f);
            const float inv = 1.f / scale;
            if (live && t == 0) p.scale[row] = scale;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int col = (i * TPR + t) * V;
                if (live && col < p.width) store_e4m3(p.y8 + o + col, s[i], inv);
            }
        }    }
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

// Blocks of an SM that the backward's registers leave room for.
template <typename T, int TPR, int NV>
constexpr int bwd_per_sm() {
    constexpr int regs = kVecOf<T> == 8 ? (NV == 1 ? 80 : 128) : (NV == 1 ? 64 : NV == 2 ? 80 : NV == 3 ? 104 : 128);
    constexpr int n = 65536 / (regs * kBlock<TPR>);
    return n < 1 ? 1 : n;
}
// The next row's loads go out before this one's reductions where registers allow.
template <typename T, int NV>
constexpr bool kBwdAhead = kVecOf<T> == 8 ? NV == 1 : NV <= 2;

// persistent: each group of TPR threads takes every (gridDim.x * groups)-th
// row and sums its rows' dw and db terms in registers; the block's sums go to its row of `part`.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(kBlock<TPR>, bwd_per_sm<T, TPR, NV>()) layernorm_bwd_kernel(BwdParams p) {
    constexpr int V = kVecOf<T>, W = kBlock<TPR> / 32;
    constexpr int G = kBlock<TPR> / TPR, ROW = TPR * NV * V;
    constexpr bool AHEAD = kBwdAhead<T, NV>;
    __shared__ float sh1[W][2], sh2[W][3];
    extern __shared__ __align__(16) float row_sh[];   // ROW weights; at the end the groups' sums
    next_grid_may_start();
    previous_grid_done();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int64_t stride = (int64_t)gridDim.x * G;
    const T *sp = (const T *)p.s, *dyp = (const T *)p.dy, *dsp = (const T *)p.dsum;
    struct Raw {
        uint4 s[NV], d[NV], u[NV];
    } cur, next;
    int64_t row = (int64_t)blockIdx.x * G + grp;
    auto load = [&](Raw &r, int64_t at) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            r.s[i] = r.d[i] = r.u[i] = make_uint4(0, 0, 0, 0);
            if (at < p.rows && col < p.width) {
                const int64_t o = at * p.width + col;
                r.s[i] = load16(sp + o);
                r.d[i] = load16(dyp + o);
                if (dsp) r.u[i] = load16(dsp + o);
            }
        }
    };
    if (AHEAD) load(cur, row);
    for (int i = threadIdx.x; i < ROW; i += kBlock<TPR>) row_sh[i] = i < p.width ? p.w[i] : 0.f;
    float2 dw[NV][V / 2], db[NV][V / 2];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < V / 2; j++) dw[i][j] = db[i][j] = make_float2(0.f, 0.f);
    __syncthreads();
    // every group of the block makes the same number of turns (the barriers)
    for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += stride, row += stride) {
        if (AHEAD) load(next, row + stride);
        else load(cur, row);
        float one[2] = {0.f, 0.f};   // sums of s and u
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float s[V], d[V], w[V];
            widen16(cur.s[i], s);
            widen16(cur.d[i], d);
            load_floats(row_sh + (i * TPR + t) * V, w);
#pragma unroll
            for (int j = 0; j < V; j++) {
                one[0] += s[j];
                one[1] = fmaf(w[j], d[j], one[1]);
            }
        }
        row_sums<TPR>(one, sh1);
        const float mean = one[0] * p.inv_width, mu = one[1] * p.inv_width;
        float two[3] = {0.f, 0.f, 0.f};   // with c = s - mean: sums of c, c^2 and u c
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if ((i * TPR + t) * V >= p.width) continue;
            float s[V], d[V], w[V];
            widen16(cur.s[i], s);
            widen16(cur.d[i], d);
            load_floats(row_sh + (i * TPR + t) * V, w);
#pragma unroll
            for (int j = 0; j < V; j++) {
                const float c = s[j] - mean;
                two[0] += c;
                two[1] = fmaf(c, c, two[1]);
                two[2] = fmaf(w[j] * d[j], c, two[2]);
            }
        }
        row_sums<TPR>(two, sh2);
        const float off = two[0] * p.inv_width;
        // rows past the last are zeros: with eps of 0 their rstd would be infinite
        const float rstd =
            row < p.rows ? rsqrtf(max_nan(fmaf(-off, off, two[1] * p.inv_width), 0.f) + p.eps) : 0.f;
        const float dot = fmaf(-off, mu, two[2] * p.inv_width) * rstd;   // mean(u xh)
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int col = (i * TPR + t) * V;
            float s[V], d[V], u[V], w[V], ds[V];
            widen16(cur.s[i], s);
            widen16(cur.d[i], d);
            widen16(cur.u[i], u);
            load_floats(row_sh + (i * TPR + t) * V, w);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float2 xh = make_float2(((s[j] - mean) - off) * rstd, ((s[j + 1] - mean) - off) * rstd);
                const float2 dd = make_float2(d[j], d[j + 1]);
                dw[i][j / 2] = fma2(dd, xh, dw[i][j / 2]);
                db[i][j / 2] = add2(db[i][j / 2], dd);
                ds[j] = fmaf(rstd, fmaf(w[j], d[j], -mu) - xh.x * dot, u[j]);
                ds[j + 1] = fmaf(rstd, fmaf(w[j + 1], d[j + 1], -mu) - xh.y * dot, u[j + 1]);
            }
            if (row < p.rows && col < p.width) store16((T *)p.ds + row * p.width + col, ds);
        }
        if (AHEAD) cur = next;
    }
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
            for (int col = threadIdx.x; col < p.width; col += kBlock<TPR>) {
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

template <typename T, int TPR, int NV>
int fwd(const FwdParams &p, int sms, void *st) {
    constexpr int per = kBlock<TPR> / TPR;
    const int64_t grid = std::min<int64_t>((p.rows + per - 1) / per, (int64_t)sms * fwd_per_sm<T, TPR, NV>());
    return launch_early(p.y8 ? layernorm_fwd_kernel<T, TPR, NV, true> : layernorm_fwd_kernel<T, TPR, NV, false>,
                        dim3((unsigned)grid), kBlock<TPR>, 0, 1, st, p);
}

template <typename T, int TPR, int NV>
int bwd(const BwdParams &p, int grid, float *dw, float *db, void *st) {
    constexpr size_t smem = (size_t)kBlock<TPR> * NV * kVecOf<T> * sizeof(float);
    static_assert(smem * bwd_per_sm<T, TPR, NV>() <= 220 * 1024, "the blocks of an SM fit its shared memory");
    const int rc = launch_early(layernorm_bwd_kernel<T, TPR, NV>, dim3((unsigned)grid), kBlock<TPR>, smem, 1, st, p);
    if (rc) return rc;
    return launch_column_sums2(p.part, grid, p.width, dw, db, st);
}

// Threads and vectors of a row of the backward, which holds dw and db: one
// bf16 vector a thread as long as 512 threads do.
template <typename T, typename F>
int by_width_bwd(int width, F f) {
    const int vecs = (width + kVecOf<T> - 1) / kVecOf<T>;
    if constexpr (kVecOf<T> == 8) {
        if (vecs > 48 && vecs <= 64) return with<64, 1>(f);
        if (vecs > 96 && vecs <= 128) return with<128, 1>(f);
        if (vecs > 192 && vecs <= 256) return with<256, 1>(f);
        if (vecs > 256 && vecs <= 512) return with<512, 1>(f);
        if (vecs > 512 && vecs <= 1024) return with<512, 2>(f);
    }
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
        constexpr int TPR = decltype(tpr)::value;
        s = Shape{kBlock<TPR> / TPR, bwd_per_sm<T, TPR, decltype(nv)::value>()};
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
        return by_width<float>(width, [&](auto tpr, auto nv) {
            return fwd<float, decltype(tpr)::value, decltype(nv)::value>(p, sms, stream);
        });
    return by_width<__nv_bfloat16>(width, [&](auto tpr, auto nv) {
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
