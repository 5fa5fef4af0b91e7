// Gated linear recurrence, the diagonal sibling of the delta rule: per
// channel c and token t of a sequence
//     h_t = a_t h_{t-1} + x_t,   a_t = exp(g_t),   y_t = h_t,
// and its gradients, from dy and the final state's gradient dhT,
//     dh_t = dy_t + q_t,   q_t = a_{t+1} dh_{t+1}  (q = dhT behind the last token),
//     dx_t = dh_t,   dg_t = dh_t a_t h_{t-1},   dh0 = a_0 dh_0.
//
// Bound by HBM: 8 bytes per bf16 element forward (x 2, g 4, y 2), 14
// backward, a handful of operations each, so every tensor goes through the
// chip once.  A channel's tokens depend on one another only through affine
// maps h -> A h + B, which compose: (A1, B1) then (A2, B2) is
// (A2 A1, A2 B1 + B2).  One warp takes 64 channels (2 per lane: rows of 128
// bytes of bf16) by kGroup = 16 tokens in registers, a CTA 8 such groups one
// behind the other, a cluster of up to 8 CTAs 8 times as many; each step of
// the cluster composes the groups' maps (shared memory inside the CTA,
// distributed shared memory between CTAs), and every group then runs its
// tokens from its own start.  So nothing is read twice and no CTA waits on
// another cluster; all sums run in a fixed order, and the result does not
// depend on timing.  The sequential part, one exchange per cluster step, is
// hidden by the other CTAs of the SM.
//
// The backward recomputes h inside each group from the state before the
// group's first token (the carry, fp32, 4 bytes per 16 tokens, that the
// forward keeps) instead of reading y, which is rounded and as large as x.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cpdr_internal.hpp"
#include "vec_io.cuh"

namespace cpdr {
namespace {

using namespace vio;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlice = 64;                  // channels of a CTA
constexpr int kTile = kWarps * kGlrGroup;   // tokens of a CTA per step
constexpr int kMaxCluster = 8;

struct Params {
    const GlrSpan *spans;
    const void *x;
    const float *g;
    const float *carry_in;      // backward
    const void *dy;             // backward
    const float *h0;            // forward: h0; backward: dhT
    void *y;                    // forward: y; backward: dx
    float *dg;                  // backward
    float *hT;                  // forward: hT; backward: dh0
    float *carry;               // forward
    int64_t L;                  // tokens per part of the zigzag layout
    int parts;                  // parts of the zigzag layout, 0 for the contiguous one
    int channels, slices;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 16 bytes into the same shared-memory place of CTA `rank` of the cluster.
__device__ __forceinline__ void store_remote(const float4 *local, uint32_t rank, float4 v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(r), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// Memory position of token `x` of a row (row coordinates).
__device__ __forceinline__ int64_t mem_of(const Params &p, int64_t x) {
    const int64_t part = x / p.L, off = x - part * p.L;
    const int64_t slot = 2 * part < p.parts ? 2 * part : 2 * (p.parts - 1 - part) + 1;
    return slot * p.L + off;
}

// Element offsets of the group's tokens: one run of consecutive rows, or, in
// the zigzag layout across a part's border, row by row.
struct Rows {
    int64_t first;      // memory row of the group's first token
    int64_t coord;      // its row coordinate (zigzag)
    int64_t base;       // memory row of the batch row
    bool run;           // rows follow one another in memory
    __device__ __forceinline__ int64_t at(const Params &p, int u) const {
        return run ? first + u : base + mem_of(p, coord + u);
    }
};

__device__ __forceinline__ Rows rows_of(const Params &p, const GlrSpan &sp, int64_t p0, int n) {
    Rows r;
    r.base = sp.base;
    r.coord = sp.start + p0;
    r.run = true;
    r.first = sp.base + r.coord;
    if (p.parts > 0 && n > 0) {
        r.first = sp.base + mem_of(p, r.coord);
        r.run = r.coord / p.L == (r.coord + n - 1) / p.L;
    }
    return r;
}

// The maps of one cluster step.  `fold` runs the incoming value through the
// maps before this group and leaves the value after the whole step in
// `carry`.  REV: groups and CTAs follow one another from the last to the first.
template <bool REV>
struct Exchange {
    float4 group[2][kWarps][32];         // (A0, B0, A1, B1) of each group's channel pair
    float4 cta[2][kMaxCluster][32];      // the same of each CTA of the cluster

    __device__ __forceinline__ float2 step(int par, int w, int lane, uint32_t rank, uint32_t nz, float2 A, float2 B,
                                           float2 &carry) {
        group[par][w][lane] = make_float4(A.x, B.x, A.y, B.y);
        __syncthreads();
        if (nz > 1) {
            if (w == 0) {
                float4 f = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
                for (int i = 0; i < kWarps; i++) {
                    const float4 m = group[par][REV ? kWarps - 1 - i : i][lane];
                    f = make_float4(m.x * f.x, fmaf(m.x, f.y, m.y), m.z * f.z, fmaf(m.z, f.w, m.w));
                }
                for (uint32_t z = 0; z < nz; z++) store_remote(&cta[par][rank][lane], z, f);
            }
            cluster_arrive();
            cluster_wait();
        }
        float2 start = carry;
        if (nz > 1) {
            float2 v = carry;
            for (uint32_t i = 0; i < nz; i++) {
                const uint32_t z = REV ? nz - 1 - i : i;
                if (z == rank) start = v;
                const float4 m = cta[par][z][lane];
                v = make_float2(fmaf(m.x, v.x, m.y), fmaf(m.z, v.y, m.w));
            }
            carry = v;
        }
        float2 v = start;
#pragma unroll
        for (int i = 0; i < kWarps; i++) {
            const int ww = REV ? kWarps - 1 - i : i;
            if (ww == w) start = v;
            const float4 m = group[par][ww][lane];
            v = make_float2(fmaf(m.x, v.x, m.y), fmaf(m.z, v.y, m.w));
        }
        if (nz == 1) carry = v;
        return start;
    }
};

// grid: (span, channel slice) items x cluster CTAs; cluster (nz, 1, 1)
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(Params p, int nz) {
    __shared__ Exchange<false> ex;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = nz > 1 ? cluster_rank() : 0u;
    const int item = blockIdx.x / nz;
    const GlrSpan sp = p.spans[item / p.slices];
    const int c = (item % p.slices) * kSlice + 2 * lane;
    const bool live = c < p.channels;
    const T *x = (const T *)p.x + c;
    const float *g = p.g + c;
    T *y = (T *)p.y + c;
    float2 carry = make_float2(0.f, 0.f);
    if (live && p.h0) carry = *reinterpret_cast<const float2 *>(p.h0 + (int64_t)sp.seq * p.channels + c);
    int par = 0;
    for (int64_t t0 = 0; t0 < sp.len; t0 += (int64_t)nz * kTile, par ^= 1) {
        const int64_t p0 = t0 + ((int64_t)rank * kWarps + w) * kGlrGroup;
        const int n = live ? (int)max((int64_t)0, min((int64_t)kGlrGroup, sp.len - p0)) : 0;
        const Rows rows = rows_of(p, sp, p0, n);
        Raw2<T> xr[kGlrGroup];
        float2 a[kGlrGroup];
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            xr[u] = Raw2<T>{};
            a[u] = make_float2(0.f, 0.f);   // exp(0) = 1: tokens past the end leave the state as it is
            if (u < n) {
                const int64_t o = rows.at(p, u) * p.channels;
                xr[u] = load2(x + o);
                a[u] = *reinterpret_cast<const float2 *>(g + o);
            }
        }
        float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            a[u] = make_float2(expf(a[u].x), expf(a[u].y));
            const float2 xv = widen(xr[u]);
            A = make_float2(A.x * a[u].x, A.y * a[u].y);
            B = make_float2(fmaf(a[u].x, B.x, xv.x), fmaf(a[u].y, B.y, xv.y));
        }
        float2 h = ex.step(par, w, lane, rank, (uint32_t)nz, A, B, carry);
        if (n > 0 && p.carry)
            *reinterpret_cast<float2 *>(p.carry + (sp.group0 + p0 / kGlrGroup) * p.channels + c) = h;
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            const float2 xv = widen(xr[u]);
            h = make_float2(fmaf(a[u].x, h.x, xv.x), fmaf(a[u].y, h.y, xv.y));
            if (u < n) store2(y + rows.at(p, u) * p.channels, h);
        }
    }
    if (live && p.hT && rank == 0 && w == 0)
        *reinterpret_cast<float2 *>(p.hT + (int64_t)sp.seq * p.channels + c) = carry;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(Params p, int nz) {
    __shared__ Exchange<true> ex;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = nz > 1 ? cluster_rank() : 0u;
    const int item = blockIdx.x / nz;
    const GlrSpan sp = p.spans[item / p.slices];
    const int c = (item % p.slices) * kSlice + 2 * lane;
    const bool live = c < p.channels;
    const T *x = (const T *)p.x + c;
    const T *dy = (const T *)p.dy + c;
    const float *g = p.g + c;
    T *dx = (T *)p.y + c;
    float *dg = p.dg + c;
    float2 carry = make_float2(0.f, 0.f);
    if (live && p.h0) carry = *reinterpret_cast<const float2 *>(p.h0 + (int64_t)sp.seq * p.channels + c);
    const int64_t step = (int64_t)nz * kTile;
    int par = 0;
    for (int64_t t0 = (sp.len - 1) / step * step; t0 >= 0 && sp.len > 0; t0 -= step, par ^= 1) {
        const int64_t p0 = t0 + ((int64_t)rank * kWarps + w) * kGlrGroup;
        const int n = live ? (int)max((int64_t)0, min((int64_t)kGlrGroup, sp.len - p0)) : 0;
        const Rows rows = rows_of(p, sp, p0, n);
        float2 a[kGlrGroup], hp[kGlrGroup];
        Raw2<T> xr[kGlrGroup], dr[kGlrGroup];
        float2 h = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            xr[u] = Raw2<T>{};
            dr[u] = Raw2<T>{};
            a[u] = make_float2(0.f, 0.f);
            if (u < n) {
                const int64_t o = rows.at(p, u) * p.channels;
                xr[u] = load2(x + o);
                a[u] = *reinterpret_cast<const float2 *>(g + o);
                dr[u] = load2(dy + o);
            }
        }
        if (n > 0) h = *reinterpret_cast<const float2 *>(p.carry_in + (sp.group0 + p0 / kGlrGroup) * p.channels + c);
        float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            a[u] = make_float2(expf(a[u].x), expf(a[u].y));
            hp[u] = h;
            const float2 xv = widen(xr[u]);
            h = make_float2(fmaf(a[u].x, h.x, xv.x), fmaf(a[u].y, h.y, xv.y));
            A = make_float2(A.x * a[u].x, A.y * a[u].y);
        }
#pragma unroll
        for (int u = kGlrGroup - 1; u >= 0; u--) {
            const float2 d = widen(dr[u]);
            B = make_float2(a[u].x * (d.x + B.x), a[u].y * (d.y + B.y));
        }
        float2 q = ex.step(par, w, lane, rank, (uint32_t)nz, A, B, carry);
#pragma unroll
        for (int u = kGlrGroup - 1; u >= 0; u--) {
            const float2 d = widen(dr[u]);
            const float2 dh = make_float2(d.x + q.x, d.y + q.y);
            q = make_float2(a[u].x * dh.x, a[u].y * dh.y);
            if (u < n) {
                const int64_t o = rows.at(p, u) * p.channels;
                store2(dx + o, dh);
                *reinterpret_cast<float2 *>(dg + o) = make_float2(q.x * hp[u].x, q.y * hp[u].y);
            }
        }
    }
    if (live && p.hT && rank == 0 && w == 0)
        *reinterpret_cast<float2 *>(p.hT + (int64_t)sp.seq * p.channels + c) = carry;
}

// One token for each row: grid (channel blocks, rows).  Rows of one slot are
// consecutive tokens of its sequence, in row order: the first of them runs
// them all, the others leave.
template <typename T>
__global__ void __launch_bounds__(kThreads)
glr_step_kernel(const T *__restrict__ x, const float *__restrict__ g, const float *state, float *state_out,
                const int32_t *__restrict__ slots, int n, int num_slots, int channels, T *y) {
    const int row = blockIdx.y;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 2;
    int slot = row;
    bool more = false;   // later rows of the same slot
    if (slots) {
        slot = slots[row];
        bool earlier = false, later = false;
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const bool same = slots[j] == slot;
            earlier |= same && j < row;
            later |= same && j > row;
        }
        if (slot < 0 || slot >= num_slots) return;
        if (__syncthreads_or(earlier)) return;
        more = __syncthreads_or(later) != 0;
    }
    if (c >= channels) return;
    const int64_t so = (int64_t)slot * channels + c;
    float2 h = *reinterpret_cast<const float2 *>(state + so);
    for (int j = row; j < n; j++) {
        if (j != row && slots[j] != slot) continue;
        const int64_t o = (int64_t)j * channels + c;
        const float2 gv = *reinterpret_cast<const float2 *>(g + o);
        const float2 xv = widen(load2(x + o));
        h = make_float2(fmaf(expf(gv.x), h.x, xv.x), fmaf(expf(gv.y), h.y, xv.y));
        store2(y + o, h);
        if (!more) break;
    }
    *reinterpret_cast<float2 *>(state_out + so) = h;
}

// CTAs of a cluster: as many as keep the items' clusters within two CTAs per
// SM, and no more than the longest sequence has tiles.
int pick_cluster(const cpdr_ctx *c, int64_t items) {
    const int64_t room = 2 * (int64_t)device_sms(c->device);
    int z = 1;
    while (z < kMaxCluster && items * 2 * z <= room && c->plan.glr_longest > (int64_t)z * kTile) z *= 2;
    return z;
}

template <typename K>
int launch(const cpdr_ctx *c, K kernel, Params p, void *stream) {
    const auto &pl = c->plan;
    p.spans = c->dev.glr_spans;
    p.L = pl.L;
    p.parts = (pl.flags & CPDR_FLAG_LAYOUT_ZIGZAG) ? pl.R : 0;
    p.slices = (p.channels + kSlice - 1) / kSlice;
    const int64_t items = (int64_t)pl.glr_spans.size() * p.slices;
    const int nz = pick_cluster(c, items);
    if (items * nz > (int64_t)0x7fffffff) return (int)cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(items * nz));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)nz;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = nz > 1 ? 1 : 0;
    return (int)cudaLaunchKernelEx(&cfg, kernel, p, nz);
}

}  // namespace

int launch_glr_fwd(const cpdr_ctx *c, const void *x, const float *g, const float *h0, int channels, void *y,
                   float *hT, float *carry, void *stream) {
    Params p{};
    p.x = x;
    p.g = g;
    p.h0 = h0;
    p.y = y;
    p.hT = hT;
    p.carry = carry;
    p.channels = channels;
    return c->plan.in_dtype == CPDR_DTYPE_F32 ? launch(c, glr_fwd_kernel<float>, p, stream)
                                              : launch(c, glr_fwd_kernel<__nv_bfloat16>, p, stream);
}

int launch_glr_bwd(const cpdr_ctx *c, const void *x, const float *g, const float *carry, const void *dy,
                   const float *dhT, int channels, void *dx, float *dg, float *dh0, void *stream) {
    Params p{};
    p.x = x;
    p.g = g;
    p.carry_in = carry;
    p.dy = dy;
    p.h0 = dhT;
    p.y = dx;
    p.dg = dg;
    p.hT = dh0;
    p.channels = channels;
    return c->plan.in_dtype == CPDR_DTYPE_F32 ? launch(c, glr_bwd_kernel<float>, p, stream)
                                              : launch(c, glr_bwd_kernel<__nv_bfloat16>, p, stream);
}

int launch_glr_step(const cpdr_ctx *c, const void *x, const float *g, const float *state, float *state_out,
                    const int32_t *slots, int n, int num_slots, int channels, void *y, void *stream) {
    if (n == 0) return 0;
    const dim3 grid((unsigned)((channels + 2 * kThreads - 1) / (2 * kThreads)), (unsigned)n);
    cudaStream_t st = (cudaStream_t)stream;
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        glr_step_kernel<float><<<grid, kThreads, 0, st>>>((const float *)x, g, state, state_out, slots, n, num_slots,
                                                          channels, (float *)y);
    else
        glr_step_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>((const __nv_bfloat16 *)x, g, state, state_out, slots,
                                                                  n, num_slots, channels, (__nv_bfloat16 *)y);
    return (int)cudaGetLastError();
}

}  // namespace cpdr
