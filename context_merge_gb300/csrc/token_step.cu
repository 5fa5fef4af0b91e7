// The serving forms of the token mixers: tokens over a pool of slots.
//
// The gated delta rule token by token over a pool of state slots: its serving
// form, which goes on from the final states that the chunk form leaves.  Per
// row, state head h and token, with S [dk, dv] the slot's state and a = exp(g)
// (one number, or one per key dim),
//     P = Diag(a) S,   D = beta (v - P^T k),   S' = P + k D^T,
//     o = scale S'^T q = scale (P^T q + (q . k) D),
// the last form because it needs no S': one pass over P gives P^T k and P^T q
// of every query head of the state, and one reduction is all that a token waits
// for.  Products and sums are fp32; o is rounded once.
//
// Bound by HBM: a state is read and written once, however many tokens of its
// sequence the call brings; it stays in registers between them.  The columns of
// S (the value dims) do not depend on one another, so a state head is cut into
// slices of 32 of them, one CTA each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cpdr_internal.hpp"
#include "launch.cuh"
#include "vec_io.cuh"

namespace cpdr {
namespace {

using namespace vio;

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kSlice = 32;   // value dims of a CTA

struct Params {
    const void *q, *k, *v, *beta;
    const float *g;
    const float *state;
    float *state_out;
    const int32_t *slots;
    void *o;
    int n, num_slots, H, G;
    float scale;
};

__device__ __forceinline__ float at(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float at(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void put(float *p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// The rows that continue one slot.  begin() tells whether `row` is the first
// of them (the others leave it to that one), next() the one behind row j.
struct Rows {
    const int32_t *slots;
    int n, slot, last;
    int base;         // next() has looked at the rows before this one, but for those of `found`
    uint32_t found;   // rows of the slot among the 32 before `base`

    // the whole block calls it; false: nothing to do
    __device__ __forceinline__ bool begin(const int32_t *s, int count, int num_slots, int row, int *shared_last) {
        slots = s;
        n = count;
        slot = last = row;
        if (!s) return true;
        if (threadIdx.x == 0) *shared_last = row;
        slot = s[row];
        bool earlier = false;
        int behind = row;
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const bool same = s[j] == slot;
            earlier |= same && j < row;
            if (same && j > behind) behind = j;
        }
        if (slot < 0 || slot >= num_slots) return false;
        if (__syncthreads_or(earlier)) return false;
        behind = __reduce_max_sync(0xffffffffu, behind);
        if ((threadIdx.x & 31) == 0 && behind > row) atomicMax(shared_last, behind);
        __syncthreads();
        last = *shared_last;
        base = row + 1;
        found = 0;
        return true;
    }
    __device__ __forceinline__ int next(int j) {
        if (j >= last) return n;
        while (!found) {
            const int i = base + (threadIdx.x & 31);
            found = __ballot_sync(0xffffffffu, i < n && slots[i] == slot);
            base += 32;
        }
        const int i = base - 32 + __ffs(found) - 1;
        found &= found - 1;
        return i;
    }
};

// [dk, dv] states.  A thread holds four columns of the slice (lane % 8) and
// every 16th row: sums over rows go over four lanes of a warp and the four warps.
// GP: query heads per round, the first round shared with P^T k.
template <typename T, int D, bool KDA, int GP>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(Params p) {
    constexpr int N = D / (4 * kWarps);           // rows of a thread
    constexpr int R = 4 * (1 + GP) + 4;           // sums of a thread: P^T k, P^T q, q . k (padded to 16 bytes)
    static_assert(GP <= 4, "q . k of a round fits four floats");
    __shared__ int shared_last;
    __shared__ __align__(16) float red[2][kWarps][8][R];
    next_grid_may_start();
    previous_grid_done();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x / (D / kSlice), col = blockIdx.x % (D / kSlice) * kSlice + (lane & 7) * 4;
    const int row = blockIdx.y;
    Rows rows;
    if (!rows.begin(p.slots, p.n, p.num_slots, row, &shared_last)) return;
    const int64_t so = ((int64_t)rows.slot * p.H + h) * D * D + col;
    const int k0 = w * 4 + (lane >> 3);           // rows k0 + 16 i
    float4 S[N];
#pragma unroll
    for (int i = 0; i < N; i++) S[i] = *reinterpret_cast<const float4 *>(p.state + so + (int64_t)(k0 + 16 * i) * D);
    const T *qp = (const T *)p.q, *kp = (const T *)p.k, *vp = (const T *)p.v, *bp = (const T *)p.beta;
    int par = 0;
    for (int j = row; j < p.n; j = rows.next(j)) {
        const int64_t hk = (int64_t)j * p.H + h, hq = (int64_t)j * p.H * p.G + (int64_t)h * p.G;
        float k[N];
#pragma unroll
        for (int i = 0; i < N; i++) k[i] = at(kp, hk * D + k0 + 16 * i);
        if (KDA) {
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float a = expf(p.g[hk * D + k0 + 16 * i]);
                S[i] = make_float4(a * S[i].x, a * S[i].y, a * S[i].z, a * S[i].w);
            }
        } else {
            const float a = expf(p.g[hk]);
#pragma unroll
            for (int i = 0; i < N; i++) S[i] = make_float4(a * S[i].x, a * S[i].y, a * S[i].z, a * S[i].w);
        }
        for (int g0 = 0; g0 < p.G; g0 += GP) {
            float r[R];
#pragma unroll
            for (int i = 0; i < R; i++) r[i] = 0.f;
            if (g0 == 0) {
#pragma unroll
                for (int i = 0; i < N; i++) {
                    r[0] = fmaf(k[i], S[i].x, r[0]);
                    r[1] = fmaf(k[i], S[i].y, r[1]);
                    r[2] = fmaf(k[i], S[i].z, r[2]);
                    r[3] = fmaf(k[i], S[i].w, r[3]);
                }
            }
#pragma unroll
            for (int g = 0; g < GP; g++) {
                if (g0 + g >= p.G) continue;
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const float q = at(qp, (hq + g0 + g) * D + k0 + 16 * i);
                    float *b = r + 4 * (1 + g);
                    b[0] = fmaf(q, S[i].x, b[0]);
                    b[1] = fmaf(q, S[i].y, b[1]);
                    b[2] = fmaf(q, S[i].z, b[2]);
                    b[3] = fmaf(q, S[i].w, b[3]);
                    r[4 * (1 + GP) + g] = fmaf(q, k[i], r[4 * (1 + GP) + g]);
                }
            }
#pragma unroll
            for (int i = 0; i < R; i++) {
                r[i] += __shfl_xor_sync(0xffffffffu, r[i], 8);
                r[i] += __shfl_xor_sync(0xffffffffu, r[i], 16);
            }
            if (lane < 8) {
#pragma unroll
                for (int i = 0; i < R; i += 4)
                    *reinterpret_cast<float4 *>(&red[par][w][lane][i]) = make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                float4 s = *reinterpret_cast<const float4 *>(&red[par][0][lane & 7][i]);
#pragma unroll
                for (int x = 1; x < kWarps; x++) {
                    const float4 y = *reinterpret_cast<const float4 *>(&red[par][x][lane & 7][i]);
                    s = make_float4(s.x + y.x, s.y + y.y, s.z + y.z, s.w + y.w);
                }
                r[i] = s.x;
                r[i + 1] = s.y;
                r[i + 2] = s.z;
                r[i + 3] = s.w;
            }
            par ^= 1;   // the next round writes the other half: its barrier is behind these reads
            float d[4] = {0.f, 0.f, 0.f, 0.f};   // the later rounds read S' itself
            if (g0 == 0) {
                const float beta = at(bp, hk);
#pragma unroll
                for (int c = 0; c < 4; c++) d[c] = beta * (at(vp, hk * D + col + c) - r[c]);
#pragma unroll
                for (int i = 0; i < N; i++)
                    S[i] = make_float4(fmaf(k[i], d[0], S[i].x), fmaf(k[i], d[1], S[i].y), fmaf(k[i], d[2], S[i].z),
                                       fmaf(k[i], d[3], S[i].w));
            }
            if (threadIdx.x < 8) {
#pragma unroll
                for (int g = 0; g < GP; g++) {
                    if (g0 + g >= p.G) continue;
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        put((T *)p.o, (hq + g0 + g) * D + col + c,
                            p.scale * fmaf(r[4 * (1 + GP) + g], d[c], r[4 * (1 + g) + c]));
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; i++) *reinterpret_cast<float4 *>(p.state_out + so + (int64_t)(k0 + 16 * i) * D) = S[i];
}

// [dv, dk] states: a row of S^T (one value dim) lies along D / 4 lanes, four
// key dims each; a warp holds 8 value dims and needs no other warp.
template <typename T, int D, bool KDA, int GP>
__global__ void __launch_bounds__(kThreads) delta_step_vfirst_kernel(Params p) {
    constexpr int L = D / 4, PER = 32 / L;        // lanes of a value dim, value dims of one load
    constexpr int N = 8 / PER;                    // value dims of a thread
    __shared__ int shared_last;
    next_grid_may_start();
    previous_grid_done();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x / (D / kSlice);
    const int v0 = blockIdx.x % (D / kSlice) * kSlice + w * 8 + lane / L, k0 = lane % L * 4;   // value dims v0 + PER i
    const int row = blockIdx.y;
    Rows rows;
    if (!rows.begin(p.slots, p.n, p.num_slots, row, &shared_last)) return;
    const int64_t so = (((int64_t)rows.slot * p.H + h) * D + v0) * D + k0;
    float4 S[N];
#pragma unroll
    for (int i = 0; i < N; i++) S[i] = *reinterpret_cast<const float4 *>(p.state + so + PER * i * D);
    const T *qp = (const T *)p.q, *kp = (const T *)p.k, *vp = (const T *)p.v, *bp = (const T *)p.beta;
    auto four = [&](const T *x, int64_t i) { return make_float4(at(x, i), at(x, i + 1), at(x, i + 2), at(x, i + 3)); };
    auto dot = [](float4 a, float4 b) { return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w))); };
    auto sum = [](float x) {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    };
    for (int j = row; j < p.n; j = rows.next(j)) {
        const int64_t hk = (int64_t)j * p.H + h, hq = (int64_t)j * p.H * p.G + (int64_t)h * p.G;
        const float4 k = four(kp, hk * D + k0);
        float4 a;
        if (KDA) {
            a = *reinterpret_cast<const float4 *>(p.g + hk * D + k0);
            a = make_float4(expf(a.x), expf(a.y), expf(a.z), expf(a.w));
        } else {
            a.x = a.y = a.z = a.w = expf(p.g[hk]);
        }
        float d[N];
        const float beta = at(bp, hk);
#pragma unroll
        for (int i = 0; i < N; i++) {
            S[i] = make_float4(a.x * S[i].x, a.y * S[i].y, a.z * S[i].z, a.w * S[i].w);
            d[i] = beta * (at(vp, hk * D + v0 + PER * i) - sum(dot(k, S[i])));
            S[i] = make_float4(fmaf(k.x, d[i], S[i].x), fmaf(k.y, d[i], S[i].y), fmaf(k.z, d[i], S[i].z),
                               fmaf(k.w, d[i], S[i].w));
        }
        for (int g = 0; g < p.G; g++) {
            const float4 q = four(qp, (hq + g) * D + k0);
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float o = sum(dot(q, S[i]));
                if (k0 == 0) put((T *)p.o, (hq + g) * D + v0 + PER * i, p.scale * o);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; i++) *reinterpret_cast<float4 *>(p.state_out + so + PER * i * D) = S[i];
}

// The causal conv's tokens: y = act(b + sum_i w_i x_i) over a slot's W - 1 kept
// inputs (oldest first) and the row's own, which then is the newest one kept.  A
// thread owns one 16-byte vector of channels, whose weights stay in registers.
struct ConvParams {
    const void *x;
    const float *weight, *bias;
    const void *state;
    void *state_out;
    const int32_t *slots;
    void *y;
    int n, num_slots, channels;
};

// as in the conv over sequences: the fast divide returns 0 once the denominator
// passes 2^126, where the exact quotient is below 1e-36
__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

// grid (channel blocks, rows)
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv1d_step_kernel(ConvParams p) {
    constexpr int V = kVecOf<T>, NW = W > 1 ? W - 1 : 1;
    __shared__ int shared_last;
    next_grid_may_start();
    previous_grid_done();
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V;
    const int row = blockIdx.y;
    Rows rows;
    if (!rows.begin(p.slots, p.n, p.num_slots, row, &shared_last)) return;
    const bool live = c < p.channels;   // the block stays whole for next()
    const int64_t so = (int64_t)rows.slot * (W - 1) * p.channels + c;
    float w[W][V], b[V];
    uint4 win[NW];
    if (live) {
#pragma unroll
        for (int i = 0; i < W - 1; i++) win[i] = load16((const T *)p.state + so + (int64_t)i * p.channels);
#pragma unroll
        for (int j = 0; j < V; j++) {
#pragma unroll
            for (int i = 0; i < W; i++) w[i][j] = p.weight[(int64_t)(c + j) * W + i];
            b[j] = p.bias ? p.bias[c + j] : 0.f;
        }
    }
    for (int j = row; j < p.n; j = rows.next(j)) {
        if (!live) continue;
        const int64_t o = (int64_t)j * p.channels + c;
        const uint4 x = load16((const T *)p.x + o);
        float z[V], t[V];
#pragma unroll
        for (int e = 0; e < V; e++) z[e] = b[e];
#pragma unroll
        for (int i = 0; i < W; i++) {
            widen16(i < W - 1 ? win[i < W - 1 ? i : 0] : x, t);
#pragma unroll
            for (int e = 0; e < V; e++) z[e] = fmaf(w[i][e], t[e], z[e]);
        }
        if (SILU) {
#pragma unroll
            for (int e = 0; e < V; e++) z[e] = silu(z[e]);
        }
        store16((T *)p.y + o, z);
#pragma unroll
        for (int i = 0; i + 1 < W - 1; i++) win[i] = win[i + 1];
        if (W > 1) win[NW - 1] = x;
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < W - 1; i++) *reinterpret_cast<uint4 *>((T *)p.state_out + so + (int64_t)i * p.channels) = win[i];
}

template <typename T, int W>
int conv_w(const ConvParams &p, bool silu, void *stream) {
    constexpr int per = kThreads * kVecOf<T>;
    const dim3 grid((unsigned)((p.channels + per - 1) / per), (unsigned)p.n);
    return launch_early(silu ? conv1d_step_kernel<T, W, true> : conv1d_step_kernel<T, W, false>, grid, kThreads, 0, 1, stream, p);
}

template <typename T>
int conv_t(const ConvParams &p, int width, bool silu, void *stream) {
    switch (width) {
        case 1: return conv_w<T, 1>(p, silu, stream);
        case 2: return conv_w<T, 2>(p, silu, stream);
        case 3: return conv_w<T, 3>(p, silu, stream);
        case 4: return conv_w<T, 4>(p, silu, stream);
        case 5: return conv_w<T, 5>(p, silu, stream);
        case 6: return conv_w<T, 6>(p, silu, stream);
        case 7: return conv_w<T, 7>(p, silu, stream);
        case 8: return conv_w<T, 8>(p, silu, stream);
        default: return (int)cudaErrorInvalidValue;
    }
}
static_assert(kMaxConvWidth == 8, "the dispatch covers widths 1..8");

template <typename T, int D, bool KDA>
int launch(const Params &p, bool vfirst, void *stream) {
    const dim3 grid((unsigned)(p.H * (D / kSlice)), (unsigned)p.n);
    if (vfirst) return launch_early(delta_step_vfirst_kernel<T, D, KDA, 1>, grid, kThreads, 0, 1, stream, p);
    return launch_early(p.G == 1   ? delta_step_kernel<T, D, KDA, 1>
                        : p.G == 2 ? delta_step_kernel<T, D, KDA, 2>
                                   : delta_step_kernel<T, D, KDA, 4>,
                        grid, kThreads, 0, 1, stream, p);
}

template <typename T>
int launch_t(const cpdr_ctx *c, const Params &p, void *stream) {
    const bool kda = c->plan.gate_kind == CPDR_GATE_PER_DIM, vf = c->plan.vfirst;
    if (c->plan.dk == 128) return kda ? launch<T, 128, true>(p, vf, stream) : launch<T, 128, false>(p, vf, stream);
    return kda ? launch<T, 64, true>(p, vf, stream) : launch<T, 64, false>(p, vf, stream);
}

}  // namespace

int launch_delta_step(const cpdr_ctx *c, const void *q, const void *k, const void *v, const void *beta, const float *g,
                      const float *state, float *state_out, const int32_t *slots, int n, int num_slots, void *o,
                      void *stream) {
    if (n == 0) return 0;
    const auto &pl = c->plan;
    const Params p{q, k, v, beta, g, state, state_out, slots, o, n, num_slots, pl.H, pl.G, pl.scale};
    return pl.in_dtype == CPDR_DTYPE_F32 ? launch_t<float>(c, p, stream) : launch_t<__nv_bfloat16>(c, p, stream);
}

int launch_conv1d_step(const cpdr_ctx *c, const void *x, const float *weight, const float *bias, const void *state,
                       void *state_out, const int32_t *slots, int n, int num_slots, int channels, int activation, void *y,
                       void *stream) {
    if (n == 0) return 0;
    const ConvParams p{x, weight, bias, state, state_out, slots, y, n, num_slots, channels};
    const int W = c->plan.conv_width;
    return c->plan.in_dtype == CPDR_DTYPE_F32 ? conv_t<float>(p, W, activation != 0, stream)
                                              : conv_t<__nv_bfloat16>(p, W, activation != 0, stream);
}

}  // namespace cpdr
