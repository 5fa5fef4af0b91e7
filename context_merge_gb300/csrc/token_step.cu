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

#include <algorithm>

#include "cpdr_internal.hpp"
#include "launch.cuh"
#include "vec_io.cuh"

namespace cpdr {
namespace {

using namespace vio;

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kSlice = 32;   // value dims of a CTA

__device__ __forceinline__ float at(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float at(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void put(float *p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// The rows of one slot: `row`, the first of them, to `last`.
struct Rows {
    const int32_t *slots;
    int n, slot, last;
    int base;         // next() has looked at the rows before this one, but for those of `found`
    uint32_t found;   // rows of the slot among the 32 before `base`

    __device__ __forceinline__ Rows(const int32_t *slots, int n, int slot, int row, int last)
        : slots(slots), n(n), slot(slot), last(last), base(row + 1), found(0) {}
    // The row behind row j, n when there is none; the whole warp calls it.
    __device__ __forceinline__ int next(int j) {
        if (j >= last) return n;
        while (!found) {
            if (base > last) return n;   // only if the slots changed meanwhile
            const int i = base + (threadIdx.x & 31);
            found = __ballot_sync(0xffffffffu, i <= last && slots[i] == slot);
            base += 32;
        }
        const int i = base - 32 + __ffs(found) - 1;
        found &= found - 1;
        return i;
    }
};

// For each of R rows and their slots: the last row of the slot, or kEarlier where a row
// before it has the slot, which that one then takes along.  The whole block calls it; `sh`
// holds R ints per warp.
constexpr int kEarlier = 0x7fffffff;
template <int R>
__device__ __forceinline__ void last_rows(const int32_t *slots, int n, const int (&slot)[R], int row, int (&last)[R],
                                          int (*sh)[R]) {
#pragma unroll
    for (int r = 0; r < R; r++) last[r] = row + r;
#pragma unroll 4
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const int s = slots[j];
#pragma unroll
        for (int r = 0; r < R; r++)
            if (s == slot[r]) last[r] = max(last[r], j < row + r ? kEarlier : j);
    }
#pragma unroll
    for (int r = 0; r < R; r++) last[r] = __reduce_max_sync(0xffffffffu, last[r]);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int r = 0; r < R; r++) sh[threadIdx.x >> 5][r] = last[r];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; w++)
#pragma unroll
        for (int r = 0; r < R; r++) last[r] = max(last[r], sh[w][r]);
}

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

// This CTA's row has a slot, and the row before has another one.
__device__ __forceinline__ bool slot_of(const Params &p, int row, int &slot) {
    slot = row;
    if (!p.slots) return true;
    slot = p.slots[row];
    const int before = row ? p.slots[row - 1] : -1;
    return slot >= 0 && slot < p.num_slots && slot != before;
}

// A token as the [dk, dv] kernel reads it: k, q and the gate's factors as pairs of the
// same value, for packed arithmetic.
template <int D, bool KDA, int GP>
struct Token {
    alignas(16) float2 k[D], q[GP][D], a[KDA ? D : 1];
    alignas(16) float v[kSlice];   // read four at a time
    float beta;
};
// What one thread fetches of it.
template <typename T, int D, bool KDA, int GP>
struct Fetch {
    T kq[GP + 1], v, beta;
    float a;
    __device__ __forceinline__ void load(const Params &p, int row, int h, int v0) {
        const int t = threadIdx.x;
        const int64_t hk = (int64_t)row * p.H + h, hq = hk * p.G;
        if (t < D) {
            kq[GP] = ((const T *)p.k)[hk * D + t];
#pragma unroll
            for (int g = 0; g < GP; g++) kq[g] = g < p.G ? ((const T *)p.q)[(hq + g) * D + t] : T(0.f);
            if (KDA) a = p.g[hk * D + t];
        }
        if (t < kSlice) v = ((const T *)p.v)[hk * D + v0 + t];
        if (t == kThreads - 1) {
            beta = ((const T *)p.beta)[hk];
            if (!KDA) a = p.g[hk];
        }
    }
    __device__ __forceinline__ void store(Token<D, KDA, GP> &s) const {
        const int t = threadIdx.x;
        if (t < D) {
            s.k[t] = both((float)kq[GP]);
#pragma unroll
            for (int g = 0; g < GP; g++) s.q[g][t] = both((float)kq[g]);
            if (KDA) s.a[t] = both(expf(a));
        }
        if (t < kSlice) s.v[t] = (float)v;
        if (t == kThreads - 1) {
            s.beta = (float)beta;
            if (!KDA) s.a[0] = both(expf(a));
        }
    }
};

// Four columns of a row.
struct Quad {
    float2 x, y;
};
__device__ __forceinline__ Quad mul(float2 a, const Quad &b) { return Quad{mul2(a, b.x), mul2(a, b.y)}; }
__device__ __forceinline__ void fma(Quad &c, float2 a, const Quad &b) {
    c.x = fma2(a, b.x, c.x);
    c.y = fma2(a, b.y, c.y);
}

// [dk, dv] states.  A thread holds four columns of the slice (lane % 8) and
// every 16th row: sums over rows go over four lanes of a warp and the four warps.
// A token's vectors are fetched by one thread per dim while the token before
// runs.  GP: query heads of the first round, which shares its reduction with P^T k.
constexpr int kStepPerSm[5] = {0, 5, 4, 0, 3};   // CTAs of an SM, by GP
template <typename T, int D, bool KDA, int GP>
__global__ void __launch_bounds__(kThreads, kStepPerSm[GP]) delta_step_kernel(Params p) {
    constexpr int N = D / (4 * kWarps);           // rows of a thread
    constexpr int R = 4 * (1 + GP) + GP;          // sums of a thread: P^T k, P^T q, q . k
    constexpr int RP = (R + 3) / 4 * 4;
    __shared__ int shared_last[kWarps][1];
    __shared__ Token<D, KDA, GP> tok[2];
    __shared__ __align__(16) float red[2][kWarps][8][RP];
    next_grid_may_start();
    previous_grid_done();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x / (D / kSlice), v0 = blockIdx.x % (D / kSlice) * kSlice, c0 = (lane & 7) * 4;
    const int row = blockIdx.y;
    Fetch<T, D, KDA, GP> f;
    f.load(p, row, h, v0);
    int slot[1], last[1];
    if (!slot_of(p, row, slot[0])) return;
    const int64_t so = ((int64_t)slot[0] * p.H + h) * D * D + v0 + c0;
    const int k0 = w * 4 + (lane >> 3);           // rows k0 + 16 i
    Quad S[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float4 x = *reinterpret_cast<const float4 *>(p.state + so + (k0 + 16 * i) * D);
        S[i] = Quad{make_float2(x.x, x.y), make_float2(x.z, x.w)};
    }
    f.store(tok[0]);
    last[0] = row;
    if (p.slots) last_rows<1>(p.slots, p.n, slot, row, last, shared_last);
    else __syncthreads();
    if (last[0] == kEarlier) return;
    Rows rows(p.slots, p.n, slot[0], row, last[0]);
    int par = 0, turn = 0;
    for (int j = row; j < p.n; turn ^= 1) {
        const int next = rows.next(j);
        if (next < p.n) f.load(p, next, h, v0);
        const Token<D, KDA, GP> &t = tok[turn];
        const int64_t hq = ((int64_t)j * p.H + h) * p.G;
        Quad a{}, b[GP];
        float qk[GP];
#pragma unroll
        for (int g = 0; g < GP; g++) {
            b[g] = Quad{};
            qk[g] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float2 k = t.k[k0 + 16 * i];
            S[i] = mul(t.a[KDA ? k0 + 16 * i : 0], S[i]);
            fma(a, k, S[i]);
#pragma unroll
            for (int g = 0; g < GP; g++) {
                const float2 q = t.q[g][k0 + 16 * i];
                fma(b[g], q, S[i]);
                qk[g] = fmaf(q.x, k.x, qk[g]);
            }
        }
        float r[RP] = {};
        auto lay = [&](int i, const Quad &x) {
            r[i] = x.x.x;
            r[i + 1] = x.x.y;
            r[i + 2] = x.y.x;
            r[i + 3] = x.y.y;
        };
        auto sum = [&](int count) {
#pragma unroll
            for (int i = 0; i < RP; i++) {
                if (i >= count) continue;
                r[i] += __shfl_xor_sync(0xffffffffu, r[i], 8);
                r[i] += __shfl_xor_sync(0xffffffffu, r[i], 16);
            }
            if (lane < 8) {
#pragma unroll
                for (int i = 0; i < RP; i += 4)
                    *reinterpret_cast<float4 *>(&red[par][w][lane][i]) = make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RP; i += 4) {
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
            par ^= 1;   // the next sum writes the other half: its barrier is behind these reads
        };
        lay(0, a);
#pragma unroll
        for (int g = 0; g < GP; g++) {
            lay(4 + 4 * g, b[g]);
            r[4 + 4 * GP + g] = qk[g];
        }
        if (next < p.n) f.store(tok[turn ^ 1]);   // read behind the sum's barrier
        sum(R);
        const float4 v = *reinterpret_cast<const float4 *>(&t.v[c0]);
        const float d[4] = {t.beta * (v.x - r[0]), t.beta * (v.y - r[1]), t.beta * (v.z - r[2]), t.beta * (v.w - r[3])};
        const Quad dq{make_float2(d[0], d[1]), make_float2(d[2], d[3])};
#pragma unroll
        for (int i = 0; i < N; i++) fma(S[i], t.k[k0 + 16 * i], dq);
        T *o = (T *)p.o + hq * D + v0 + c0;
        if (threadIdx.x < 8) {
#pragma unroll
            for (int g = 0; g < GP; g++)
                if (g < p.G) {
#pragma unroll
                    for (int c = 0; c < 4; c++) put(o, g * D + c, p.scale * fmaf(r[4 + 4 * GP + g], d[c], r[4 + 4 * g + c]));
                }
        }
        // the query heads behind the first GP read S' itself
        for (int g0 = GP; g0 < p.G; g0 += GP) {
#pragma unroll
            for (int g = 0; g < GP; g++) {
                b[g] = Quad{};
                if (g0 + g < p.G) {
#pragma unroll
                    for (int i = 0; i < N; i++)
                        fma(b[g], both(at((const T *)p.q, (hq + g0 + g) * D + k0 + 16 * i)), S[i]);
                }
                lay(4 * g, b[g]);
            }
            sum(4 * GP);
            if (threadIdx.x < 8) {
#pragma unroll
                for (int g = 0; g < GP; g++)
                    if (g0 + g < p.G) {
#pragma unroll
                        for (int c = 0; c < 4; c++) put(o, (int64_t)(g0 + g) * D + c, p.scale * r[4 * g + c]);
                    }
            }
        }
        __syncthreads();   // the token has been read before its place is filled again
        j = next;
    }
#pragma unroll
    for (int i = 0; i < N; i++)
        *reinterpret_cast<float4 *>(p.state_out + so + (k0 + 16 * i) * D) = make_float4(S[i].x.x, S[i].x.y, S[i].y.x, S[i].y.y);
}

// Four neighbouring values as loaded.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
    float4 r;
    __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ Quad wide() const { return Quad{make_float2(r.x, r.y), make_float2(r.z, r.w)}; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ Quad wide() const {
        return Quad{widen(Raw2<__nv_bfloat16>{r.x}), widen(Raw2<__nv_bfloat16>{r.y})};
    }
};

__device__ __forceinline__ float dot(const Quad &a, const Quad &b) {
    const float2 s = fma2(a.x, b.x, mul2(a.y, b.y));
    return s.x + s.y;
}

// x[i] of the lanes of a group of L are summed over it, value i ending up in
// its lanes with lane / (L / N) = i: each step hands half of the values over.
template <int N, int L>
__device__ __forceinline__ float spread_sum(float (&x)[N]) {
    const int lane = threadIdx.x & 31;
    int o = L / 2;
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < N / 2; i++) {
            if (i >= n) continue;
            const float give = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    for (; o > 0; o /= 2) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    return x[0];
}

// [dv, dk] states: a row of S^T (one value dim) lies along D / 4 lanes, four
// key dims each; a warp holds 8 value dims and needs no other warp.
constexpr int kVfirstPerSm[5] = {0, 5, 5, 0, 4};
template <typename T, int D, bool KDA, int GP>
__global__ void __launch_bounds__(kThreads, kVfirstPerSm[GP]) delta_step_vfirst_kernel(Params p) {
    constexpr int L = D / 4, PER = 32 / L;        // lanes of a value dim, value dims of one load
    constexpr int N = 8 / PER;                    // value dims of a thread
    __shared__ int shared_last[kWarps][1];
    next_grid_may_start();
    previous_grid_done();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x / (D / kSlice);
    const int v0 = blockIdx.x % (D / kSlice) * kSlice + w * 8 + lane / L, k0 = lane % L * 4;   // value dims v0 + PER i
    const int own = lane % L / (L / N);           // the value dim whose sums end up here
    const int row = blockIdx.y;
    // one token as loaded, fetched while the one before runs
    struct Raw {
        Raw4<T> k, q[GP];
        T v, beta;
        float4 a;
    } f;
    auto load = [&](int j) {
        const int64_t hk = (int64_t)j * p.H + h, hq = hk * p.G;
        f.k.load((const T *)p.k + hk * D + k0);
#pragma unroll
        for (int g = 0; g < GP; g++) f.q[g].load((const T *)p.q + (hq + (g < p.G ? g : 0)) * D + k0);
        f.v = ((const T *)p.v)[hk * D + v0 + PER * own];
        f.beta = ((const T *)p.beta)[hk];
        if (KDA) f.a = *reinterpret_cast<const float4 *>(p.g + hk * D + k0);
        else f.a.x = p.g[hk];
    };
    load(row);
    int slot[1], last[1];
    if (!slot_of(p, row, slot[0])) return;
    const int64_t so = (((int64_t)slot[0] * p.H + h) * D + v0) * D + k0;
    Quad S[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float4 x = *reinterpret_cast<const float4 *>(p.state + so + PER * i * D);
        S[i] = Quad{make_float2(x.x, x.y), make_float2(x.z, x.w)};
    }
    last[0] = row;
    if (p.slots) last_rows<1>(p.slots, p.n, slot, row, last, shared_last);
    if (last[0] == kEarlier) return;
    Rows rows(p.slots, p.n, slot[0], row, last[0]);
    for (int j = row; j < p.n;) {
        const int64_t hq = ((int64_t)j * p.H + h) * p.G;
        const Quad k = f.k.wide();
        Quad q[GP], a;
#pragma unroll
        for (int g = 0; g < GP; g++) q[g] = f.q[g].wide();
        if (KDA) {
            a.x = make_float2(expf(f.a.x), expf(f.a.y));
            a.y = make_float2(expf(f.a.z), expf(f.a.w));
        } else {
            a.x = a.y = both(expf(f.a.x));
        }
        const float v = (float)f.v, beta = (float)f.beta;
        const int next = rows.next(j);
        if (next < p.n) load(next);
        float x[N], y[GP][N], qk[GP];
#pragma unroll
        for (int i = 0; i < N; i++) {
            S[i] = Quad{mul2(a.x, S[i].x), mul2(a.y, S[i].y)};
            x[i] = dot(k, S[i]);
#pragma unroll
            for (int g = 0; g < GP; g++) y[g][i] = dot(q[g], S[i]);
        }
#pragma unroll
        for (int g = 0; g < GP; g++) qk[g] = dot(q[g], k);
#pragma unroll
        for (int o = L / 2; o > 0; o /= 2)
#pragma unroll
            for (int g = 0; g < GP; g++) qk[g] += __shfl_xor_sync(0xffffffffu, qk[g], o);
        const float d = beta * (v - spread_sum<N, L>(x));
        T *out = (T *)p.o + hq * D + v0 + PER * own;
        const bool writes = lane % (L / N) == 0;
#pragma unroll
        for (int g = 0; g < GP; g++) {
            const float o = p.scale * fmaf(qk[g], d, spread_sum<N, L>(y[g]));
            if (writes && g < p.G) put(out, g * D, o);
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float2 e = both(__shfl_sync(0xffffffffu, d, lane / L * L + i * (L / N)));
            S[i].x = fma2(k.x, e, S[i].x);
            S[i].y = fma2(k.y, e, S[i].y);
        }
        // the query heads behind the first GP read S' itself
        for (int g = GP; g < p.G; g++) {
            Raw4<T> r;
            r.load((const T *)p.q + (hq + g) * D + k0);
            const Quad qx = r.wide();
#pragma unroll
            for (int i = 0; i < N; i++) x[i] = dot(qx, S[i]);
            const float o = p.scale * spread_sum<N, L>(x);
            if (writes) put(out, (int64_t)g * D, o);
        }
        j = next;
    }
#pragma unroll
    for (int i = 0; i < N; i++)
        *reinterpret_cast<float4 *>(p.state_out + so + PER * i * D) = make_float4(S[i].x.x, S[i].x.y, S[i].y.x, S[i].y.y);
}

// The causal conv's tokens: y = act(b + sum_i w_i x_i) over a slot's W - 1 kept
// inputs (oldest first) and the row's own, which then is the newest one kept.  A
// thread owns one 16-byte vector of channels; its weights stay in registers
// for the rows of its block.
struct ConvParams {
    const void *x;
    const float *weight, *bias;
    const void *state;
    void *state_out;
    const int32_t *slots;
    void *y;
    int n, num_slots, channels, groups;   // groups of kConvRows rows for a block
};
constexpr int kConvRows = 2;   // rows whose loads a thread has in flight

// as in the conv over sequences: the fast divide returns 0 once the denominator
// passes 2^126, where the exact quotient is below 1e-36
__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

// grid (channel blocks, blocks of rows)
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv1d_step_kernel(ConvParams p) {
    constexpr int V = kVecOf<T>, NW = W > 1 ? W - 1 : 1, R = kConvRows;
    __shared__ int shared_last[2][kWarps][R];
    next_grid_may_start();
    previous_grid_done();
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V;
    const bool live = c < p.channels;   // the block stays whole for the rows' search
    const T *state = (const T *)p.state + c;
    const int64_t C = p.channels;
    float w[W * V], b[V];   // w[V' W + i]: as they lie
    if (live) {
#pragma unroll
        for (int i = 0; i < W * V; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p.weight + (int64_t)c * W + i);
            w[i] = x.x;
            w[i + 1] = x.y;
            w[i + 2] = x.z;
            w[i + 3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 x = p.bias ? *reinterpret_cast<const float4 *>(p.bias + c + j) : make_float4(0.f, 0.f, 0.f, 0.f);
            b[j] = x.x;
            b[j + 1] = x.y;
            b[j + 2] = x.z;
            b[j + 3] = x.w;
        }
    }
    // y of row j, and the window moved on
    auto token = [&](int j, uint4 (&win)[NW], const uint4 &x) {
        float z[V], t[V];
#pragma unroll
        for (int e = 0; e < V; e++) z[e] = b[e];
#pragma unroll
        for (int i = 0; i < W; i++) {
            widen16(i < W - 1 ? win[i < W - 1 ? i : 0] : x, t);
#pragma unroll
            for (int e = 0; e < V; e++) z[e] = fmaf(w[e * W + i], t[e], z[e]);
        }
        if (SILU) {
#pragma unroll
            for (int e = 0; e < V; e++) z[e] = silu(z[e]);
        }
        store16((T *)p.y + j * C + c, z);
#pragma unroll
        for (int i = 0; i + 1 < W - 1; i++) win[i] = win[i + 1];
        if (W > 1) win[NW - 1] = x;
    };
    for (int i = 0; i < p.groups; i++) {
        const int row = (blockIdx.y * p.groups + i) * R;
        if (row >= p.n) break;
        int slot[R], last[R];
        bool used[R];
        uint4 win[R][NW], x[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            last[r] = row + r;
            slot[r] = row + r >= p.n ? -1 : p.slots ? p.slots[row + r] : row + r;
            used[r] = slot[r] >= 0 && slot[r] < p.num_slots;
            x[r] = make_uint4(0, 0, 0, 0);
            if (live && used[r]) {
                x[r] = load16((const T *)p.x + (row + r) * C + c);
#pragma unroll
                for (int u = 0; u < W - 1; u++) win[r][u] = load16(state + ((int64_t)slot[r] * (W - 1) + u) * C);
            }
        }
        if (p.slots) last_rows<R>(p.slots, p.n, slot, row, last, shared_last[i & 1]);
#pragma unroll
        for (int r = 0; r < R; r++) {
            if (!used[r] || last[r] == kEarlier) continue;
            Rows rows(p.slots, p.n, slot[r], row + r, last[r]);
            for (int j = row + r; j < p.n; j = rows.next(j)) {
                if (!live) continue;
                token(j, win[r], j == row + r ? x[r] : load16((const T *)p.x + j * C + c));
            }
            if (live) {
#pragma unroll
                for (int u = 0; u < W - 1; u++)
                    *reinterpret_cast<uint4 *>((T *)p.state_out + ((int64_t)slot[r] * (W - 1) + u) * C + c) = win[r][u];
            }
        }
    }
}

template <typename T, int W>
int conv_w(ConvParams p, bool silu, int sms, void *stream) {
    constexpr int per = kThreads * kVecOf<T>;
    const int blocks = (p.channels + per - 1) / per, groups = (p.n + kConvRows - 1) / kConvRows;
    // several groups of rows for a block, which reads the weights once for them, as long as there are blocks for the GPU
    p.groups = (int)std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)groups * blocks / (4 * sms)));
    const dim3 grid((unsigned)blocks, (unsigned)((groups + p.groups - 1) / p.groups));
    return launch_early(silu ? conv1d_step_kernel<T, W, true> : conv1d_step_kernel<T, W, false>, grid, kThreads, 0, 1, stream, p);
}

template <typename T>
int conv_t(const ConvParams &p, int width, bool silu, int sms, void *stream) {
    switch (width) {
        case 1: return conv_w<T, 1>(p, silu, sms, stream);
        case 2: return conv_w<T, 2>(p, silu, sms, stream);
        case 3: return conv_w<T, 3>(p, silu, sms, stream);
        case 4: return conv_w<T, 4>(p, silu, sms, stream);
        case 5: return conv_w<T, 5>(p, silu, sms, stream);
        case 6: return conv_w<T, 6>(p, silu, sms, stream);
        case 7: return conv_w<T, 7>(p, silu, sms, stream);
        case 8: return conv_w<T, 8>(p, silu, sms, stream);
        default: return (int)cudaErrorInvalidValue;
    }
}
static_assert(kMaxConvWidth == 8, "the dispatch covers widths 1..8");

template <typename T, int D, bool KDA, int GP>
int launch_g(const Params &p, bool vfirst, void *stream) {
    const dim3 grid((unsigned)(p.H * (D / kSlice)), (unsigned)p.n);
    return launch_early(vfirst ? delta_step_vfirst_kernel<T, D, KDA, GP> : delta_step_kernel<T, D, KDA, GP>, grid, kThreads, 0, 1,
                        stream, p);
}

template <typename T, int D, bool KDA>
int launch(const Params &p, bool vfirst, void *stream) {
    if (p.G == 1) return launch_g<T, D, KDA, 1>(p, vfirst, stream);
    if (p.G == 2) return launch_g<T, D, KDA, 2>(p, vfirst, stream);
    return launch_g<T, D, KDA, 4>(p, vfirst, stream);
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
    const ConvParams p{x, weight, bias, state, state_out, slots, y, n, num_slots, channels, 1};
    const int W = c->plan.conv_width, sms = device_sms(c->device);
    return c->plan.in_dtype == CPDR_DTYPE_F32 ? conv_t<float>(p, W, activation != 0, sms, stream)
                                              : conv_t<__nv_bfloat16>(p, W, activation != 0, sms, stream);
}

}  // namespace cpdr
