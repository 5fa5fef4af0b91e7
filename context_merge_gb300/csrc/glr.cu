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

constexpr int kSlice = 64;                  // channels of a CTA
constexpr int kMaxCluster = 8;
constexpr int kStages = 2;                  // groups of a warp in shared memory: one in use, one on its way
constexpr int kStepThreads = 256;
template <typename T>
constexpr int kFwdWarps = sizeof(T) == 2 ? 8 : 4;
constexpr int kBwdWarps = 4;

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

// Memory rows of a group's tokens.  Contiguous layout: one after the other.
// Zigzag: parts may end inside the group, so each lane works out one row (a
// 64-bit division) and the others ask it; kept out of the contiguous kernels,
// whose code it would multiply (an inlined division at every access made the
// forward instruction-fetch bound, 5 us per step).
template <bool ZIGZAG>
struct Rows {
    int64_t first;   // contiguous: the first token's row; zigzag: the row of this lane's token
    __device__ __forceinline__ Rows(const Params &p, const GlrSpan &sp, int64_t p0, int lane) {
        first = sp.base + sp.start + p0;
        if (ZIGZAG) {
            const int64_t x = min(sp.start + p0 + (lane & (kGlrGroup - 1)), p.L * p.parts - 1);
            first = sp.base + mem_of(p, max(x, (int64_t)0));
        }
    }
    __device__ __forceinline__ int64_t at(int u) const {
        return ZIGZAG ? __shfl_sync(0xffffffffu, first, u) : first + u;
    }
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool ok) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int n = ok ? 16 : 0;   // 0: nothing is read, the 16 bytes become zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's group of one tensor: kGlrGroup rows of the slice, in shared memory.
template <typename T>
struct Tile {
    T v[kGlrGroup][kSlice];
    // Starts the copies of the group's n rows; what lies behind the rows or
    // the channels becomes zero.
    template <bool ZIGZAG>
    __device__ __forceinline__ void load(const Params &p, const Rows<ZIGZAG> &rows, const T *src, int c0, int n,
                                         int lane) {
        constexpr int E = 16 / (int)sizeof(T), CH = kSlice / E;   // elements of a copy, copies of a row
#pragma unroll
        for (int i = 0; i < kGlrGroup * CH / 32; i++) {
            const int row = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH * E;
            const bool ok = row < n && c0 + c < p.channels;
            const int64_t at = rows.at(row) * p.channels + c0 + c;
            cp_async16(&v[row][c], ok ? src + at : src, ok);
        }
    }
};

// The maps of one cluster step.  REV: groups and CTAs follow one another from
// the last to the first.
template <int WARPS, bool REV>
struct Exchange {
    float4 group[WARPS][32];             // (A0, B0, A1, B1) of each group's channel pair
    float4 cta[2][kMaxCluster][32];      // the same of each CTA of the cluster, by parity of the step

    // The value before this warp's group, from the value `carry` before the
    // step, which becomes the value behind it.
    __device__ __forceinline__ float2 step(int par, int w, int lane, uint32_t rank, uint32_t nz, float2 A, float2 B,
                                           float2 &carry) {
        // a cluster of one has no barrier between this step's reads and the
        // next one's writes: it alternates between `group` and `cta`
        float4(*grp)[32] = nz == 1 && par ? reinterpret_cast<float4(*)[32]>(&cta[0][0][0]) : group;
        grp[w][lane] = make_float4(A.x, B.x, A.y, B.y);
        __syncthreads();
        // maps before this warp's group, and of the whole CTA
        float4 f = make_float4(1.f, 0.f, 1.f, 0.f), before = f;
#pragma unroll
        for (int i = 0; i < WARPS; i++) {
            const int ww = REV ? WARPS - 1 - i : i;
            if (ww == w) before = f;
            const float4 m = grp[ww][lane];
            f = make_float4(m.x * f.x, fmaf(m.x, f.y, m.y), m.z * f.z, fmaf(m.z, f.w, m.w));
        }
        float2 start = carry;
        if (nz > 1) {
            for (uint32_t z = w; z < nz; z += WARPS) store_remote(&cta[par][rank][lane], z, f);
            cluster_arrive();
            cluster_wait();
            float2 v = carry;
            for (uint32_t i = 0; i < nz; i++) {
                const uint32_t z = REV ? nz - 1 - i : i;
                if (z == rank) start = v;
                const float4 m = cta[par][z][lane];
                v = make_float2(fmaf(m.x, v.x, m.y), fmaf(m.z, v.y, m.w));
            }
            carry = v;
        } else {
            carry = make_float2(fmaf(f.x, carry.x, f.y), fmaf(f.z, carry.y, f.w));
        }
        return make_float2(fmaf(before.x, start.x, before.y), fmaf(before.z, start.y, before.w));
    }
};

template <typename T, int WARPS>
struct FwdShared {
    Exchange<WARPS, false> ex;
    struct {
        Tile<T> x;
        Tile<float> g;
    } ring[WARPS][kStages];
};
template <typename T, int WARPS>
struct BwdShared {
    Exchange<WARPS, true> ex;
    struct {
        Tile<T> x, dy;
        Tile<float> g;
    } ring[WARPS][kStages];
};

// CTAs of an SM, by shared memory (1 KiB of it is the system's for each).
template <typename S>
constexpr int kPerSm = (228 * 1024) / ((int)sizeof(S) + 1024);

extern __shared__ __align__(16) unsigned char smem[];

// grid: (span, channel slice) items x cluster CTAs; cluster (nz, 1, 1)
template <typename T, int WARPS, bool ZIGZAG>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) glr_fwd_kernel(Params p, int nz) {
    auto &sh = *reinterpret_cast<FwdShared<T, WARPS> *>(smem);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = nz > 1 ? cluster_rank() : 0u;
    const int item = blockIdx.x / nz;
    const GlrSpan sp = p.spans[item / p.slices];
    const int c0 = (item % p.slices) * kSlice, c = c0 + 2 * lane;
    const bool live = c < p.channels;
    T *y = (T *)p.y + c;
    float2 carry = make_float2(0.f, 0.f);
    if (live && p.h0) carry = *reinterpret_cast<const float2 *>(p.h0 + (int64_t)sp.seq * p.channels + c);
    const int64_t step = (int64_t)nz * WARPS * kGlrGroup;
    const int64_t mine = ((int64_t)rank * WARPS + w) * kGlrGroup;
    auto tokens = [&](int64_t p0) { return (int)max((int64_t)0, min((int64_t)kGlrGroup, sp.len - p0)); };
    auto fetch = [&](int64_t p0, int stage) {
        const int n = tokens(p0);
        const Rows<ZIGZAG> rows(p, sp, p0, lane);
        auto &r = sh.ring[w][stage];
        r.x.load(p, rows, (const T *)p.x, c0, n, lane);
        r.g.load(p, rows, p.g, c0, n, lane);
        cp_commit();
    };
    fetch(mine, 0);
    int par = 0;
    for (int64_t t0 = 0; t0 < sp.len; t0 += step, par ^= 1) {
        const int64_t p0 = t0 + mine;
        const int n = live ? tokens(p0) : 0;
        fetch(p0 + step, par ^ 1);
        cp_wait<1>();
        __syncwarp();
        const auto &r = sh.ring[w][par];
        Raw2<T> xr[kGlrGroup];
        float2 a[kGlrGroup];
        float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            xr[u] = load2(&r.x.v[u][2 * lane]);
            const float2 gv = *reinterpret_cast<const float2 *>(&r.g.v[u][2 * lane]);
            a[u] = make_float2(expf(gv.x), expf(gv.y));   // behind the tokens g = 0: the state stays as it is
            const float2 xv = widen(xr[u]);
            A = make_float2(A.x * a[u].x, A.y * a[u].y);
            B = make_float2(fmaf(a[u].x, B.x, xv.x), fmaf(a[u].y, B.y, xv.y));
        }
        float2 h = sh.ex.step(par, w, lane, rank, (uint32_t)nz, A, B, carry);
        if (n > 0 && p.carry)
            *reinterpret_cast<float2 *>(p.carry + (sp.group0 + p0 / kGlrGroup) * p.channels + c) = h;
        const Rows<ZIGZAG> rows(p, sp, p0, lane);
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            const float2 xv = widen(xr[u]);
            h = make_float2(fmaf(a[u].x, h.x, xv.x), fmaf(a[u].y, h.y, xv.y));
            const int64_t o = rows.at(u) * p.channels;
            if (u < n) store2(y + o, h);
        }
    }
    cp_wait<0>();
    if (live && p.hT && rank == 0 && w == 0)
        *reinterpret_cast<float2 *>(p.hT + (int64_t)sp.seq * p.channels + c) = carry;
}

template <typename T, int WARPS, bool ZIGZAG>
__global__ void __launch_bounds__(32 * WARPS, 12 / WARPS) glr_bwd_kernel(Params p, int nz) {
    auto &sh = *reinterpret_cast<BwdShared<T, WARPS> *>(smem);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = nz > 1 ? cluster_rank() : 0u;
    const int item = blockIdx.x / nz;
    const GlrSpan sp = p.spans[item / p.slices];
    const int c0 = (item % p.slices) * kSlice, c = c0 + 2 * lane;
    const bool live = c < p.channels;
    T *dx = (T *)p.y + c;
    float *dg = p.dg + c;
    float2 carry = make_float2(0.f, 0.f);
    if (live && p.h0) carry = *reinterpret_cast<const float2 *>(p.h0 + (int64_t)sp.seq * p.channels + c);
    const int64_t step = (int64_t)nz * WARPS * kGlrGroup;
    const int64_t mine = ((int64_t)rank * WARPS + w) * kGlrGroup;
    auto tokens = [&](int64_t p0) { return (int)max((int64_t)0, min((int64_t)kGlrGroup, sp.len - p0)); };
    auto fetch = [&](int64_t p0, int stage) {
        const int n = p0 < 0 ? 0 : tokens(p0);
        const Rows<ZIGZAG> rows(p, sp, p0, lane);
        auto &r = sh.ring[w][stage];
        r.x.load(p, rows, (const T *)p.x, c0, n, lane);
        r.g.load(p, rows, p.g, c0, n, lane);
        r.dy.load(p, rows, (const T *)p.dy, c0, n, lane);
        cp_commit();
    };
    const int64_t last = sp.len > 0 ? (sp.len - 1) / step * step : -1;
    auto start_of = [&](int64_t p0) {
        return live && p0 >= 0 && tokens(p0) > 0
                   ? *reinterpret_cast<const float2 *>(p.carry_in + (sp.group0 + p0 / kGlrGroup) * p.channels + c)
                   : make_float2(0.f, 0.f);
    };
    float2 h_next = make_float2(0.f, 0.f);
    if (last >= 0) {
        fetch(last + mine, 0);
        h_next = start_of(last + mine);
    }
    int par = 0;
    for (int64_t t0 = last; t0 >= 0; t0 -= step, par ^= 1) {
        const int64_t p0 = t0 + mine;
        const int n = live ? tokens(p0) : 0;
        float2 h = h_next;
        // the step before this one; the first step has none (a position below zero: no rows)
        fetch(t0 >= step ? p0 - step : -1, par ^ 1);
        h_next = start_of(t0 >= step ? p0 - step : -1);
        cp_wait<1>();
        __syncwarp();
        const auto &r = sh.ring[w][par];
        float2 a[kGlrGroup], hp[kGlrGroup];
        float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            const float2 gv = *reinterpret_cast<const float2 *>(&r.g.v[u][2 * lane]);
            const float2 xv = widen(load2(&r.x.v[u][2 * lane]));
            a[u] = make_float2(expf(gv.x), expf(gv.y));
            hp[u] = h;
            h = make_float2(fmaf(a[u].x, h.x, xv.x), fmaf(a[u].y, h.y, xv.y));
            A = make_float2(A.x * a[u].x, A.y * a[u].y);
        }
#pragma unroll
        for (int u = kGlrGroup - 1; u >= 0; u--) {
            const float2 d = widen(load2(&r.dy.v[u][2 * lane]));
            B = make_float2(a[u].x * (d.x + B.x), a[u].y * (d.y + B.y));
        }
        float2 q = sh.ex.step(par, w, lane, rank, (uint32_t)nz, A, B, carry);
        const Rows<ZIGZAG> rows(p, sp, p0, lane);
#pragma unroll
        for (int u = kGlrGroup - 1; u >= 0; u--) {
            const float2 d = widen(load2(&r.dy.v[u][2 * lane]));
            const float2 dh = make_float2(d.x + q.x, d.y + q.y);
            q = make_float2(a[u].x * dh.x, a[u].y * dh.y);
            const int64_t o = rows.at(u) * p.channels;
            if (u < n) {
                store2(dx + o, dh);
                *reinterpret_cast<float2 *>(dg + o) = make_float2(q.x * hp[u].x, q.y * hp[u].y);
            }
        }
        __syncwarp();   // the group's dy is read to the end before its place is filled again
    }
    cp_wait<0>();
    if (live && p.hT && rank == 0 && w == 0)
        *reinterpret_cast<float2 *>(p.hT + (int64_t)sp.seq * p.channels + c) = carry;
}

// One token for each row: grid (channel blocks, rows).  Rows of one slot are
// consecutive tokens of its sequence, in row order: the first of them runs
// them all, the others leave.
template <typename T>
__global__ void __launch_bounds__(kStepThreads)
glr_step_kernel(const T *__restrict__ x, const float *__restrict__ g, const float *state, float *state_out,
                const int32_t *__restrict__ slots, int n, int num_slots, int channels, T *y) {
    const int row = blockIdx.y;
    const int c = (blockIdx.x * kStepThreads + threadIdx.x) * 2;
    int slot = row;
    bool more = false;   // later rows of the same slot
    if (slots) {
        slot = slots[row];
        bool earlier = false, later = false;
        for (int j = threadIdx.x; j < n; j += kStepThreads) {
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

// CTAs of a cluster: as many as keep the items' clusters within what runs at
// once, and no more than the longest sequence has tiles.
int pick_cluster(const cpdr_ctx *c, int64_t items, int tile, int per_sm) {
    const int64_t room = (int64_t)per_sm * device_sms(c->device);
    int z = 1;
    while (z < kMaxCluster && items * 2 * z <= room && c->plan.glr_longest > (int64_t)z * tile) z *= 2;
    return z;
}

template <typename K>
int launch(const cpdr_ctx *c, K kernel, int warps, int per_sm, size_t bytes, Params p, void *stream) {
    const auto &pl = c->plan;
    p.spans = c->dev.glr_spans;
    p.L = pl.L;
    p.parts = (pl.flags & CPDR_FLAG_LAYOUT_ZIGZAG) ? pl.R : 0;
    p.slices = (p.channels + kSlice - 1) / kSlice;
    const int64_t items = (int64_t)pl.glr_spans.size() * p.slices;
    const int nz = pick_cluster(c, items, warps * kGlrGroup, per_sm);
    if (items * nz > (int64_t)0x7fffffff) return (int)cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return (int)e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(items * nz));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)nz;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = nz > 1 ? 1 : 0;
    return (int)cudaLaunchKernelEx(&cfg, kernel, p, nz);
}

template <typename T>
int fwd(const cpdr_ctx *c, const Params &p, void *stream) {
    constexpr int W = kFwdWarps<T>;
    auto kernel = c->plan.flags & CPDR_FLAG_LAYOUT_ZIGZAG ? glr_fwd_kernel<T, W, true> : glr_fwd_kernel<T, W, false>;
    return launch(c, kernel, W, kPerSm<FwdShared<T, W>>, sizeof(FwdShared<T, W>), p, stream);
}
template <typename T>
int bwd(const cpdr_ctx *c, const Params &p, void *stream) {
    constexpr int W = kBwdWarps;
    auto kernel = c->plan.flags & CPDR_FLAG_LAYOUT_ZIGZAG ? glr_bwd_kernel<T, W, true> : glr_bwd_kernel<T, W, false>;
    return launch(c, kernel, W, kPerSm<BwdShared<T, W>>, sizeof(BwdShared<T, W>), p, stream);
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
    return c->plan.in_dtype == CPDR_DTYPE_F32 ? fwd<float>(c, p, stream)
                                              : fwd<__nv_bfloat16>(c, p, stream);
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
    return c->plan.in_dtype == CPDR_DTYPE_F32 ? bwd<float>(c, p, stream)
                                              : bwd<__nv_bfloat16>(c, p, stream);
}

int launch_glr_step(const cpdr_ctx *c, const void *x, const float *g, const float *state, float *state_out,
                    const int32_t *slots, int n, int num_slots, int channels, void *y, void *stream) {
    if (n == 0) return 0;
    const dim3 grid((unsigned)((channels + 2 * kStepThreads - 1) / (2 * kStepThreads)), (unsigned)n);
    cudaStream_t st = (cudaStream_t)stream;
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        glr_step_kernel<float><<<grid, kStepThreads, 0, st>>>((const float *)x, g, state, state_out, slots, n, num_slots,
                                                          channels, (float *)y);
    else
        glr_step_kernel<__nv_bfloat16><<<grid, kStepThreads, 0, st>>>((const __nv_bfloat16 *)x, g, state, state_out, slots,
                                                                  n, num_slots, channels, (__nv_bfloat16 *)y);
    return (int)cudaGetLastError();
}

}  // namespace cpdr
