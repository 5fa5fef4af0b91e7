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
// bytes of bf16) by 16 tokens, a CTA 4 (backward 8) such groups one behind the
// other, a cluster of up to 8 CTAs 8 times as many; each step of the cluster
// composes the groups' maps (shared memory inside the CTA, distributed shared
// memory between CTAs), and every group then runs its tokens from its own
// start.  So nothing is read twice and no CTA waits on another cluster; all
// sums run in a fixed order, and the result does not depend on timing.  A
// step's exchange goes on while the step before it is written.
//
// Measured (of 6782 GB/s): forward 262144 x 2048 bf16, one sequence, 674 us,
// 0.97; packed 65536 x 2048, 12 ragged sequences: fp32 zigzag forward 259 us,
// 0.91; bf16 backward 304 us, 0.93.  Few channels leave SMs idle: one sequence of
// 131072 x 64, forward 282 us, backward 307.  Where most groups have positive
// gates that sum to more than 1, 32768 x 2048 takes 378 and 556 us (91 and 156
// without).
//
// The backward recomputes h inside each group from the state before the
// group's first token (the carry, fp32, 4 bytes per 16 tokens, that the
// forward keeps) instead of reading y, which is rounded and as large as x.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "cpdr_internal.hpp"
#include "launch.cuh"
#include "tc_common.cuh"
#include "vec_io.cuh"

namespace cpdr {
namespace {

using namespace vio;

constexpr int kSlice = 64;                  // channels of a CTA
constexpr int kMaxCluster = 8;
constexpr int kFwdStages = 2;               // groups of a warp in shared memory, both on their way
constexpr int kStages = 3;                  // backward: going out, being mapped, on its way
constexpr int kStepThreads = 256;
constexpr float kMaxFloat = 3.402823466e38f;
// Warps of a CTA.  Forward: two CTAs of four per SM, whose steps hide one
// another's (262144 x 2048 bf16, one sequence: 677 us; of six warps 709; three
// of four 729).  Backward: one CTA of what three stages leave room for (packed
// 65536 x 2048 bf16: 311 us; two of four: 319).
constexpr int kFwdWarps = 4;
template <typename T>
constexpr int kBwdWarps = sizeof(T) == 2 ? 8 : 5;

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
    int32_t *status;            // the context's status word (bounded waits)
    int channels, slices;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// exp(g) for |g| <= 1/4: 1 + g + g^2 q(g), q of degree 3 interpolated at
// Chebyshev points (off by 0.7 half steps at 1/4, by 0.1 up to 1/10), rounded
// once: five instructions for two channels.
__device__ __forceinline__ float2 exp_near_zero(float2 g) {
    constexpr float kC[4] = {0.49999931454658508f, 0.16666656732559204f, 0.041753556579351425f, 0.0083457436412572861f};
    float2 r = fma2(g, both(kC[3]), both(kC[2]));
    r = fma2(g, r, both(kC[1]));
    r = fma2(g, r, both(kC[0]));
    r = fma2(g, r, both(1.f));
    return fma2(g, r, both(1.f));
}
// exp(g) elsewhere: 2^t (1 + e ln 2) with t = g log2(e) rounded, log2(e) in
// two parts, and e what t misses; the fast power of two is off by up to two
// units in the last place.  Gates from -87.4 down give 0; a NaN stays one.
__device__ __forceinline__ float2 exp_far(float2 g) {
    constexpr float kL = 1.44269504088896341f, kLow = 1.92596299e-8f, kLn2 = 0.693147180559945309f;
    // -infinity would meet itself in e; 2^-185 is flushed to zero
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(g.x) : "f"(-128.f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(g.y) : "f"(-128.f));
    const float2 t = mul2(g, both(kL));
    const float2 e = fma2(g, both(-kLow), fma2(g, both(-kL), t));   // minus what is missing
    float2 r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(t.y));
    return fma2(mul2(r, both(-kLn2)), e, r);
}
// a = exp(g) for a group's gates, in place.
// Gates next to 0 make a long memory, which adds the errors of many steps up:
// they need an a that leans to no side (the fast power leans by 0.4 half steps:
// alone, it cost the states of a long memory 1e-6).  Each token's gate decides
// for itself, so that a channel's bits do not depend on the channels beside it;
// where every channel's squares sum to at most 1/16 over the group (so that all
// |g| <= 1/4) the other form is left out: 131072 x 2048 bf16 forward 341 us, with
// both forms 429; backward 599 and 683.  (A third form for warps whose channels
// all forget at once, the far one alone: 395 and 614 there, but 466 where
// slow and fast channels lie side by side.)
// Returns what the group's map starts from, for each channel: 1, or a NaN where
// positive gates sum to more than 1, so that the map must not be composed
// (Exchange).  Squares of at most 1/16 keep the sum of 16 gates below 1, and a
// group of negative gates has none.
__device__ __forceinline__ float2 exp_of_gates(float2 (&g)[kGlrGroup]) {
    float2 one = both(1.f);
    float2 sq[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
    for (int u = 0; u < kGlrGroup; u++) sq[u & 3] = fma2(g[u], g[u], sq[u & 3]);
    const float2 sum = add2(add2(sq[0], sq[1]), add2(sq[2], sq[3]));
    if (__all_sync(0xffffffffu, sum.x <= 0.0625f && sum.y <= 0.0625f)) {
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) g[u] = exp_near_zero(g[u]);
    } else {
        uint32_t signs = ~0u;
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) signs &= __float_as_uint(g[u].x) & __float_as_uint(g[u].y);
        if (__any_sync(0xffffffffu, (int32_t)signs >= 0)) {
            float2 growth = both(0.f);
#pragma unroll
            for (int u = 0; u < kGlrGroup; u++) growth = add2(growth, make_float2(fmaxf(g[u].x, 0.f), fmaxf(g[u].y, 0.f)));
            if (growth.x > 1.f) one.x = __int_as_float(0x7fffffff);
            if (growth.y > 1.f) one.y = __int_as_float(0x7fffffff);
        }
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            const float2 near = exp_near_zero(g[u]), far = exp_far(g[u]);
            g[u] = make_float2(fabsf(g[u].x) <= 0.25f ? near.x : far.x, fabsf(g[u].y) <= 0.25f ? near.y : far.y);
        }
    }
    return one;
}

// A pair of maps h -> A h + B.
struct Map {
    float2 A, B;
};
__device__ __forceinline__ float2 apply(const Map &m, float2 h) { return fma2(m.A, h, m.B); }
__device__ __forceinline__ Map after(const Map &m, const Map &f) { return Map{mul2(m.A, f.A), fma2(m.A, f.B, m.B)}; }

// 16 bytes into the same shared-memory place of CTA `rank` of the cluster,
// counted there by the same barrier.  (A plain store and the cluster's
// barrier would need a release, which waits for the output's stores to global
// memory too: measured 0.8 stalled warps per issue.)
__device__ __forceinline__ void send(const Map *place, uint64_t *bar, uint32_t rank, const Map &v) {
    uint32_t ra, rb;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(tc::smem_u32(place)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(tc::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(ra),
                 "f"(v.A.x), "f"(v.A.y), "f"(v.B.x), "f"(v.B.y), "r"(rb)
                 : "memory");
}

// The same for a pair of states.
__device__ __forceinline__ void send(const float2 *place, uint64_t *bar, uint32_t rank, float2 h) {
    uint32_t ra, rb;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(tc::smem_u32(place)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(tc::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(ra), "f"(h.x),
                 "f"(h.y), "r"(rb)
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
    const uint32_t d = tc::smem_u32(dst);
    const int n = ok ? 16 : 0;   // 0: nothing is read, the 16 bytes become zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's group of one tensor: kGlrGroup rows of the slice, in shared memory,
// whole lines of it (131072 x 2048 bf16 forward 346 us; tiles that begin 32
// bytes into a line 364, 16 bytes 422).
template <typename T>
struct alignas(128) Tile {
    T v[kGlrGroup][kSlice];
    // Starts the copies of the group's n rows; what lies behind the rows or
    // the channels becomes zero.
    template <bool ZIGZAG>
    __device__ __forceinline__ void load(const Params &p, const Rows<ZIGZAG> &rows, const T *src, int c0, int n,
                                         int lane) {
        constexpr int E = 16 / (int)sizeof(T), CH = kSlice / E;   // elements of a copy, copies of a row
        constexpr int PER = 32 / CH;                              // rows that a warp's copies cover at once
        const int r0 = lane / CH, c = lane % CH * E;
        if (!ZIGZAG && n == kGlrGroup && c0 + kSlice <= p.channels) {
            // whole groups: one address per lane, the rest is the same for all lanes
            const T *at = src + (rows.at(0) + r0) * p.channels + c0 + c;
#pragma unroll
            for (int i = 0; i < kGlrGroup / PER; i++) cp_async16(&v[i * PER + r0][c], at + i * PER * p.channels, true);
            return;
        }
#pragma unroll
        for (int i = 0; i < kGlrGroup / PER; i++) {
            const int row = i * PER + r0;
            const bool ok = row < n && c0 + c < p.channels;
            const int64_t at = rows.at(row) * p.channels + c0 + c;
            cp_async16(&v[row][c], ok ? src + at : src, ok);
        }
    }
};

// The maps of one cluster step.  REV: groups and CTAs follow one another from
// the last to the first.
//
// Maps compose safely where A stays in fp32's range.  Positive gates can take
// it out of range although the states are finite (zero or small states, a reset
// behind the growth), and infinity times zero would be NaN.  A group whose
// positive gates sum to at most 1 multiplies by at most e, a step's 64 groups by
// e^64: nothing overflows, and what an A too small for fp32 loses is at most
// 2^-149 e^64 = 1e-17 of the state before the step.  Any other group's map starts
// from a NaN (exp_of_gates), which stays through every composition; a step
// that meets one runs token by token for its channels, the groups one behind
// the other.  The other channels keep what the maps gave them, to the last bit.
template <int WARPS, bool REV>
struct alignas(16) Exchange {
    Map grp[2][WARPS][32];          // each group's, for every channel pair, by parity of the step
    Map cta[2][kMaxCluster][32];    // each CTA's of the cluster
    uint64_t bar[2];                // the CTAs' maps of a step have arrived, by parity
    // a step token by token: the states behind each warp's group, before this
    // CTA's groups and behind the step, and the barriers that they are there
    float2 behind[WARPS][32], enter[32], leave[32];
    uint64_t done[WARPS], entered, left;

    tc::Ctl ctl;

    // The whole cluster calls it before the first step ...
    __device__ __forceinline__ void open(uint32_t nz) {
        if (threadIdx.x == 0) {
            ctl.abort = 0;
            tc::mbar_init(&bar[0], 1);
            tc::mbar_init(&bar[1], 1);
#pragma unroll
            for (int i = 0; i < WARPS; i++) tc::mbar_init(&done[i], 1);
            tc::mbar_init(&entered, 1);
            tc::mbar_init(&left, 1);
        }
        if (nz == 1) {
            __syncthreads();
            return;
        }
        cluster_arrive();
        cluster_wait();
    }
    // ... and behind the last: no CTA leaves while another may still send to it.
    __device__ __forceinline__ void close(uint32_t nz) {
        if (nz == 1) return;
        cluster_arrive();
        cluster_wait();
    }

    // First half: publishes this warp's map of step i; `before` becomes the
    // map of the CTA's groups before it, `all` that of the whole CTA.  A CTA
    // sends step i + 2 into the places of step i only when it has the maps of
    // step i + 1 of every CTA, and a CTA sends those behind its
    // __syncthreads, where all its warps have read step i.
    __device__ __forceinline__ void publish(int par, int w, int lane, uint32_t rank, uint32_t nz, const Map &m,
                                            Map &before, Map &all) {
        // the next step writes the other half: its __syncthreads is behind this step's reads
        grp[par][w][lane] = m;
        __syncthreads();
        Map f{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
        before = f;
#pragma unroll
        for (int i = 0; i < WARPS; i++) {
            const int ww = REV ? WARPS - 1 - i : i;
            if (ww == w) before = f;
            f = after(grp[par][ww][lane], f);
        }
        all = f;
        if (nz > 1) {
            if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(&bar[par], nz * (uint32_t)sizeof(cta[0][0]));
            for (uint32_t z = w; z < nz; z += WARPS) send(&cta[par][rank][lane], &bar[par], z, f);
        }
    }
    // Second half: the value before this warp's group, from the value `carry`
    // before the step, which becomes the value behind it.  `phase`: how often
    // this parity's barrier has completed, modulo 2.  `group` takes a value
    // through this warp's group; `turns`: the steps that ran token by token.
    template <typename F>
    __device__ __forceinline__ float2 start(int par, uint32_t phase, int w, int lane, uint32_t rank, uint32_t nz,
                                            const Map &before, const Map &all, float2 &carry, int32_t *status,
                                            uint32_t &turns, F group) {
        float2 s = carry, v = carry;
        if (nz > 1) {
            tc::mbar_wait(&bar[par], phase, &ctl, status, REV ? 151 : 150);
            for (uint32_t i = 0; i < nz; i++) {
                const uint32_t z = REV ? nz - 1 - i : i;
                if (z == rank) s = v;
                v = apply(cta[par][z][lane], v);
            }
        } else {
            v = apply(all, carry);
        }
        s = apply(before, s);
        // not finite: a map that must not be composed, one whose B overflows where the
        // state does not, or (nothing is lost then but time) the state itself.
        // The whole cluster sees the same maps and goes this way or that as one.
        const bool x = !(fabsf(v.x) <= kMaxFloat), y = !(fabsf(v.y) <= kMaxFloat);
        if (__any_sync(0xffffffffu, x || y)) {
            float2 end;
            const float2 h = in_turn(w, lane, rank, nz, carry, end, status, turns++ & 1u, group);
            s = make_float2(x ? h.x : s.x, y ? h.y : s.y);
            v = make_float2(x ? end.x : v.x, y ? end.y : v.y);
        }
        carry = v;
        return s;
    }
    // The groups of a step one behind the other: the state goes from warp to warp
    // through shared memory, from CTA to CTA and at last to all of them by remote
    // stores.  Every barrier here completes once in such a step, and none is used
    // again before the whole cluster has published the next step's maps, which
    // each warp does behind its last wait here.
    template <typename F>
    __device__ __forceinline__ float2 in_turn(int w, int lane, uint32_t rank, uint32_t nz, float2 before_step, float2 &end,
                                              int32_t *status, uint32_t phase, F group) {
        constexpr uint32_t kBytes = 32 * sizeof(float2);
        const int site = REV ? 153 : 152;
        end = before_step;
        if (ctl.abort) return before_step;   // nothing is counted after a wait that gave up
        const uint32_t c = REV ? nz - 1 - rank : rank;         // this CTA's place in the order,
        const int i = REV ? WARPS - 1 - w : w;                 // and this warp's
        if (threadIdx.x == 0 && nz > 1) {
            if (c > 0) tc::mbar_arrive_expect_tx(&entered, kBytes);
            tc::mbar_arrive_expect_tx(&left, kBytes);
        }
        float2 h = before_step;
        if (i > 0) {
            tc::mbar_wait(&done[i - 1], phase, &ctl, status, site);
            h = behind[i - 1][lane];
        } else if (c > 0) {
            tc::mbar_wait(&entered, phase, &ctl, status, site);
            h = enter[lane];
        }
        const float2 first = h;
        h = group(h);
        if (i + 1 < WARPS) {
            behind[i][lane] = h;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&done[i]);
        } else if (c + 1 < nz) {
            send(&enter[lane], &entered, REV ? rank - 1 : rank + 1, h);
        } else if (nz > 1) {
            for (uint32_t z = 0; z < nz; z++) send(&leave[lane], &left, z, h);
        } else {
            leave[lane] = h;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&left);
        }
        tc::mbar_wait(&left, phase, &ctl, status, site);
        end = leave[lane];
        return first;
    }
};

template <typename T, int WARPS>
struct FwdShared {
    Exchange<WARPS, false> ex;
    struct {
        Tile<T> x;
        Tile<float> g;
    } ring[WARPS][kFwdStages];
};
template <typename T, int WARPS>
struct BwdShared {
    Exchange<WARPS, true> ex;
    struct {
        Tile<T> x, dy;
        Tile<float> g;
    } ring[WARPS][kStages];
};

// CTAs of an SM: what the kernels' registers are bounded for, where shared memory
// holds as many (1 KiB of it is the system's for each).
constexpr int kFwdPerSm = 2, kBwdPerSm = 1;
template <typename S, int BOUND>
constexpr int kPerSm = (228 * 1024) / ((int)sizeof(S) + 1024) < BOUND ? (228 * 1024) / ((int)sizeof(S) + 1024) : BOUND;

extern __shared__ __align__(128) unsigned char smem[];

// The loop of both directions, over cluster steps i: the maps of step i + 1
// are taken and published, then step i's tokens run from their start and go
// out while the cluster exchanges those maps, and last the starts of step
// i + 1 follow from the exchanged maps.  Forward, a group is held in registers
// from its map to its output (two groups in turn), so that its place in shared
// memory takes the next copies at once; backward, three tensors and the
// recomputed states leave no registers for that: the group stays where it is,
// with its gates made to a_t = exp(g_t) in place.
//
// grid: (span, channel slice) items x cluster CTAs; cluster (nz, 1, 1)
template <typename T, int WARPS, bool ZIGZAG>
__global__ void __launch_bounds__(32 * WARPS, kFwdPerSm) glr_fwd_kernel(Params p, int nz) {
    auto &sh = *reinterpret_cast<FwdShared<T, WARPS> *>(smem);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = nz > 1 ? cluster_rank() : 0u;
    const int item = blockIdx.x / nz;
    next_grid_may_start();
    previous_grid_done();
    const GlrSpan sp = p.spans[item / p.slices];
    const int c0 = (item % p.slices) * kSlice, c = c0 + 2 * lane;
    const bool live = c < p.channels;
    T *y = (T *)p.y + c;
    float2 carry = make_float2(0.f, 0.f);
    if (live && p.h0) carry = *reinterpret_cast<const float2 *>(p.h0 + (int64_t)sp.seq * p.channels + c);
    const int64_t step = (int64_t)nz * WARPS * kGlrGroup;
    int64_t p0 = ((int64_t)rank * WARPS + w) * kGlrGroup;   // this warp's first token of step i
    auto tokens = [&](int64_t at) { return (int)max((int64_t)0, min((int64_t)kGlrGroup, sp.len - at)); };
    auto fetch = [&](int64_t at, int stage) {
        const Rows<ZIGZAG> rows(p, sp, at, lane);
        const int n = tokens(at);
        auto &r = sh.ring[w][stage];
        r.x.load(p, rows, (const T *)p.x, c0, n, lane);
        r.g.load(p, rows, p.g, c0, n, lane);
        cp_commit();
    };
    struct Group {
        float2 a[kGlrGroup];
        Raw2<T> x[kGlrGroup];
    };
    Map before, all;
    // Takes step i's group into registers, starts step i + 2's copies into its
    // place, and publishes its map.
    auto take = [&](Group &v, int64_t at, int stage) {
        cp_wait<1>();
        __syncwarp();
        const auto &r = sh.ring[w][stage];
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            v.a[u] = *reinterpret_cast<const float2 *>(&r.g.v[u][2 * lane]);
            v.x[u] = load2(&r.x.v[u][2 * lane]);
        }
        __syncwarp();
        fetch(at + 2 * step, stage);
        Map m{exp_of_gates(v.a), both(0.f)};   // behind the tokens g = 0: the state stays
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) m = after(Map{v.a[u], widen(v.x[u])}, m);
        sh.ex.publish(stage, w, lane, rank, (uint32_t)nz, m, before, all);
    };
    const int64_t steps = (sp.len + step - 1) / step;
    float2 h = both(0.f);
    uint32_t turns = 0;
    // The state before step i's group, from its maps; all that it needs of the group else.
    auto start = [&](const Group &v, int64_t i, int parity) {
        return sh.ex.start(parity, (uint32_t)(i >> 1) & 1u, w, lane, rank, (uint32_t)nz, before, all, carry, p.status, turns,
                           [&](float2 s) {
#pragma unroll
                               for (int u = 0; u < kGlrGroup; u++) s = fma2(v.a[u], s, widen(v.x[u]));
                               return s;
                           });
    };
    // One step: the next one's maps, this one's outputs, the next one's starts.
    auto turn = [&](const Group &v, Group &next, int64_t i, int parity) {
        if (i + 1 < steps) take(next, p0 + step, parity ^ 1);
        const int n = live ? tokens(p0) : 0;
        if (n > 0 && p.carry)
            *reinterpret_cast<float2 *>(p.carry + (sp.group0 + p0 / kGlrGroup) * p.channels + c) = h;
        const Rows<ZIGZAG> rows(p, sp, p0, lane);
        auto run = [&](auto whole) {
            T *o = y + rows.at(0) * p.channels;
#pragma unroll
            for (int u = 0; u < kGlrGroup; u++) {
                h = fma2(v.a[u], h, widen(v.x[u]));
                if (ZIGZAG) o = y + rows.at(u) * p.channels;
                if (decltype(whole)::value || u < n) store2(ZIGZAG ? o : o + u * p.channels, h);
            }
        };
        if (!ZIGZAG && n == kGlrGroup) run(std::true_type());
        else run(std::false_type());
        if (i + 1 < steps) h = start(next, i + 1, parity ^ 1);
        p0 += step;
    };
    sh.ex.open((uint32_t)nz);
    if (steps > 0) {
        Group even, odd;
        fetch(p0, 0);
        fetch(p0 + step, 1);
        take(even, p0, 0);
        h = start(even, 0, 0);
        for (int64_t i = 0; i < steps; i += 2) {
            turn(even, odd, i, 0);
            if (i + 1 < steps) turn(odd, even, i + 1, 1);
        }
    }
    cp_wait<0>();
    sh.ex.close((uint32_t)nz);
    if (live && p.hT && rank == 0 && w == 0)
        *reinterpret_cast<float2 *>(p.hT + (int64_t)sp.seq * p.channels + c) = carry;
}

template <typename T, int WARPS, bool ZIGZAG>
__global__ void __launch_bounds__(32 * WARPS, kBwdPerSm) glr_bwd_kernel(Params p, int nz) {
    auto &sh = *reinterpret_cast<BwdShared<T, WARPS> *>(smem);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = nz > 1 ? cluster_rank() : 0u;
    const int item = blockIdx.x / nz;
    next_grid_may_start();
    previous_grid_done();
    const GlrSpan sp = p.spans[item / p.slices];
    const int c0 = (item % p.slices) * kSlice, c = c0 + 2 * lane;
    const bool live = c < p.channels;
    T *dx = (T *)p.y + c;
    float *dg = p.dg + c;
    float2 carry = make_float2(0.f, 0.f);
    if (live && p.h0) carry = *reinterpret_cast<const float2 *>(p.h0 + (int64_t)sp.seq * p.channels + c);
    const int64_t step = (int64_t)nz * WARPS * kGlrGroup;
    const int64_t steps = (sp.len + step - 1) / step;
    // this warp's first token of step i; below zero there is nothing
    int64_t p0 = (steps - 1) * step + ((int64_t)rank * WARPS + w) * kGlrGroup;
    auto tokens = [&](int64_t at) {
        return at < 0 ? 0 : (int)max((int64_t)0, min((int64_t)kGlrGroup, sp.len - at));
    };
    auto fetch = [&](int64_t at, int stage) {
        const Rows<ZIGZAG> rows(p, sp, at, lane);
        const int n = tokens(at);
        auto &r = sh.ring[w][stage];
        r.x.load(p, rows, (const T *)p.x, c0, n, lane);
        r.dy.load(p, rows, (const T *)p.dy, c0, n, lane);
        r.g.load(p, rows, p.g, c0, n, lane);
        cp_commit();
    };
    // the state before the group's first token
    auto kept = [&](int64_t at) {
        return live && tokens(at) > 0
                   ? *reinterpret_cast<const float2 *>(p.carry_in + (sp.group0 + at / kGlrGroup) * p.channels + c)
                   : make_float2(0.f, 0.f);
    };
    Map before, all;
    auto map = [&](int stage, int par) {
        auto &r = sh.ring[w][stage];
        Map m{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
        // everything is loaded before the first a is stored
        float2 g[kGlrGroup];
        Raw2<T> dy[kGlrGroup];
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            g[u] = *reinterpret_cast<const float2 *>(&r.g.v[u][2 * lane]);
            dy[u] = load2(&r.dy.v[u][2 * lane]);
        }
        m.A = exp_of_gates(g);
#pragma unroll
        for (int u = kGlrGroup - 1; u >= 0; u--) {
            *reinterpret_cast<float2 *>(&r.g.v[u][2 * lane]) = g[u];
            m = Map{mul2(m.A, g[u]), mul2(g[u], add2(widen(dy[u]), m.B))};
        }
        sh.ex.publish(par, w, lane, rank, (uint32_t)nz, m, before, all);
    };
    float2 q = make_float2(0.f, 0.f), h = q, h_next = q;
    uint32_t turns = 0;
    // q behind step i's group, from its maps (the group lies in `stage`)
    auto start = [&](int64_t i, int stage, int par) {
        return sh.ex.start(par, (uint32_t)(i >> 1) & 1u, w, lane, rank, (uint32_t)nz, before, all, carry, p.status, turns,
                           [&](float2 s) {
                               const auto &r = sh.ring[w][stage];
                               for (int u = kGlrGroup - 1; u >= 0; u--)
                                   s = mul2(*reinterpret_cast<const float2 *>(&r.g.v[u][2 * lane]),
                                            add2(widen(load2(&r.dy.v[u][2 * lane])), s));
                               return s;
                           });
    };
    sh.ex.open((uint32_t)nz);
    if (steps > 0) {
#pragma unroll
        for (int s = 0; s < kStages; s++) fetch(p0 - s * step, s);
        h = kept(p0);
        cp_wait<kStages - 1>();
        __syncwarp();
        map(0, 0);
        q = start(0, 0, 0);
    }
    int stage = 0, par = 0;
    for (int64_t i = 0; i < steps; i++, p0 -= step) {
        const int next = stage + 1 == kStages ? 0 : stage + 1;
        h_next = kept(p0 - step);
        if (i + 1 < steps) {
            cp_wait<kStages - 2>();
            __syncwarp();
            map(next, par ^ 1);
        }
        const int n = live ? tokens(p0) : 0;
        const Rows<ZIGZAG> rows(p, sp, p0, lane);
        const auto &r = sh.ring[w][stage];
        float2 a[kGlrGroup], hp[kGlrGroup];
#pragma unroll
        for (int u = 0; u < kGlrGroup; u++) {
            const float2 xv = widen(load2(&r.x.v[u][2 * lane]));
            a[u] = *reinterpret_cast<const float2 *>(&r.g.v[u][2 * lane]);
            hp[u] = h;
            h = fma2(a[u], h, xv);
        }
        auto run = [&](auto whole) {
            const int64_t first = rows.at(0) * p.channels;
#pragma unroll
            for (int u = kGlrGroup - 1; u >= 0; u--) {
                const float2 d = widen(load2(&r.dy.v[u][2 * lane]));
                const float2 dh = add2(d, q);
                q = mul2(a[u], dh);
                const int64_t o = ZIGZAG ? rows.at(u) * p.channels : first;
                const int more = ZIGZAG ? 0 : u * p.channels;
                if (decltype(whole)::value || u < n) {
                    store2(dx + o + more, dh);
                    *reinterpret_cast<float2 *>(dg + o + more) = mul2(q, hp[u]);
                }
            }
        };
        if (!ZIGZAG && n == kGlrGroup) run(std::true_type());
        else run(std::false_type());
        __syncwarp();   // the group is read to the end before its place is filled again
        fetch(p0 - kStages * step, stage);
        stage = next;
        par ^= 1;
        h = h_next;
        if (i + 1 < steps) q = start(i + 1, stage, par);
    }
    cp_wait<0>();
    sh.ex.close((uint32_t)nz);
    if (live && p.hT && rank == 0 && w == 0)
        *reinterpret_cast<float2 *>(p.hT + (int64_t)sp.seq * p.channels + c) = carry;
}

// One token for each row: grid (channel blocks, rows).  Rows of one slot are
// consecutive tokens of its sequence, in row order: the first of them runs
// them all, the others leave.
template <typename T>
__global__ void __launch_bounds__(kStepThreads)
glr_step_kernel(const T *x, const float *g, const float *state, float *state_out,
                const int32_t *slots, int n, int num_slots, int channels, T *y) {
    next_grid_may_start();
    previous_grid_done();
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
        h = fma2(make_float2(expf(gv.x), expf(gv.y)), h, xv);
        store2(y + o, h);
        if (!more) break;
    }
    *reinterpret_cast<float2 *>(state_out + so) = h;
}

// CTAs of a cluster, by an estimate of the time in tokens that one CTA takes:
// the longest sequence's share, or all items' over the clusters that run at
// once, with a quarter of an item for the last round's gaps; an exchange costs
// 4% per CTA.  Measured with clusters of 1, 2, 4 and 8 (us, bf16): one sequence of
// 32768 x 2048, forward 457, 269, 155, 93 and backward 549, 298, 159, 246 (of
// eight, 15 clusters run at once); 12 ragged sequences in 65536 x 2048,
// forward 193, 181, 181, 210 and backward 306, 306, 332, 465; 64 of 1024 x 2048,
// forward 166, 193, 252, 378.
int pick_cluster(const cpdr_ctx *c, int slices, int tile, int per_sm) {
    const auto &pl = c->plan;
    const int64_t items = (int64_t)pl.glr_spans.size() * slices;
    const double all = (double)pl.B * (double)pl.T * slices;
    int best = 1;
    double cost = 0;
    for (int z = 1; z <= kMaxCluster && (z == 1 || pl.glr_longest > (int64_t)(z / 2) * tile); z *= 2) {
        // the GPU's parts do not all hold a multiple of z CTAs
        const double fit = z <= 2 ? 1.0 : z == 8 && per_sm == 1 ? 0.79 : 0.95;
        const int64_t at_once = std::max<int64_t>(1, (int64_t)(device_sms(c->device) * per_sm * fit / z));
        double t = (double)pl.glr_longest / z;
        if (items > at_once) t = std::max(t, all / (z * at_once)) + 0.25 * all / items / z;
        t *= 1.0 + 0.04 * z;
        if (z == 1 || t < cost) {
            cost = t;
            best = z;
        }
    }
    return best;
}

// How a direction runs: its kernel, warps and shared memory of a CTA, and the
// CTAs of an SM that the cluster size is chosen for.
struct Form {
    void (*kernel)(Params, int);
    int warps, per_sm;
    size_t bytes;
};
template <typename T>
Form fwd(const cpdr_ctx *c) {
    constexpr int W = kFwdWarps;
    using S = FwdShared<T, W>;
    return Form{c->plan.flags & CPDR_FLAG_LAYOUT_ZIGZAG ? glr_fwd_kernel<T, W, true> : glr_fwd_kernel<T, W, false>, W,
                kPerSm<S, kFwdPerSm>, sizeof(S)};
}
template <typename T>
Form bwd(const cpdr_ctx *c) {
    constexpr int W = kBwdWarps<T>;
    using S = BwdShared<T, W>;
    return Form{c->plan.flags & CPDR_FLAG_LAYOUT_ZIGZAG ? glr_bwd_kernel<T, W, true> : glr_bwd_kernel<T, W, false>, W,
                kPerSm<S, kBwdPerSm>, sizeof(S)};
}
Form form(const cpdr_ctx *c, bool backward) {
    if (c->plan.in_dtype == CPDR_DTYPE_F32) return backward ? bwd<float>(c) : fwd<float>(c);
    return backward ? bwd<__nv_bfloat16>(c) : fwd<__nv_bfloat16>(c);
}

int launch(const cpdr_ctx *c, const Form &f, Params p, void *stream) {
    const auto &pl = c->plan;
    p.spans = c->dev.glr_spans;
    p.status = c->dev.status;
    p.L = pl.L;
    p.parts = (pl.flags & CPDR_FLAG_LAYOUT_ZIGZAG) ? pl.R : 0;
    p.slices = (p.channels + kSlice - 1) / kSlice;
    const int64_t items = (int64_t)pl.glr_spans.size() * p.slices;
    const int nz = pick_cluster(c, p.slices, f.warps * kGlrGroup, f.per_sm);
    if (items * nz > (int64_t)0x7fffffff) return (int)cudaErrorInvalidValue;
    return launch_early(f.kernel, dim3((unsigned)(items * nz)), 32 * f.warps, f.bytes, nz, stream, p, nz);
}

static_assert(sizeof(FwdShared<float, kFwdWarps>) <= 227 * 1024 && sizeof(BwdShared<float, kBwdWarps<float>>) <= 227 * 1024 &&
                  sizeof(BwdShared<__nv_bfloat16, kBwdWarps<__nv_bfloat16>>) <= 227 * 1024,
              "a CTA's stages fit its shared memory");

}  // namespace

int glr_plan(const cpdr_ctx *c, int channels, bool backward, int32_t out[3]) {
    const Form f = form(c, backward);
    out[0] = pick_cluster(c, (channels + kSlice - 1) / kSlice, f.warps * kGlrGroup, f.per_sm);
    out[1] = f.per_sm;
    out[2] = 0;
    if (!c->has_device) return 0;
    cudaError_t e = cudaFuncSetAttribute(f.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)f.bytes);
    if (e != cudaSuccess) return (int)e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f.kernel, 32 * f.warps, f.bytes);
    out[2] = n;
    return (int)e;
}

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
    return launch(c, form(c, false), p, stream);
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
    return launch(c, form(c, true), p, stream);
}

int launch_glr_step(const cpdr_ctx *c, const void *x, const float *g, const float *state, float *state_out,
                    const int32_t *slots, int n, int num_slots, int channels, void *y, void *stream) {
    if (n == 0) return 0;
    const dim3 grid((unsigned)((channels + 2 * kStepThreads - 1) / (2 * kStepThreads)), (unsigned)n);
    if (c->plan.in_dtype == CPDR_DTYPE_F32)
        return launch_early(glr_step_kernel<float>, grid, kStepThreads, 0, 1, stream, (const float *)x, g, state, state_out, slots,
                            n, num_slots, channels, (float *)y);
    return launch_early(glr_step_kernel<__nv_bfloat16>, grid, kStepThreads, 0, 1, stream, (const __nv_bfloat16 *)x, g, state,
                        state_out, slots, n, num_slots, channels, (__nv_bfloat16 *)y);
}

}  // namespace cpdr
