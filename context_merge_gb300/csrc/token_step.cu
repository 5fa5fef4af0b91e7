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
// sequence the call brings and in whatever order; it stays in registers between them.  The columns of
// S (the value dims) do not depend on one another, so a state head is cut into
// slices of them, one CTA each, and a CTA's into its warps'.  No warp waits for another one
// inside a token: sums that went through shared memory and a barrier (four warps
// to 32 value dims) took 166 us where these take 157, and 97 with drafted tokens
// instead of 35.
//
// Measured, bf16, d = 128, in graphs: 512 sequences of 16 states 159 us (6.8 TB/s,
// the measured copy's rate; [dv, dk] states the same), 61 of 32 states with per-dim gates 43 us (6.0
// TB/s), one of 16 states 3.7 us (latency).  1 to 8 drafted tokens of 48
// sequences, 32 query heads on 16 states: 35 to 36 us where the states' bytes take 16: bound by
// instructions (70% of the issue slots), 250 a token and warp.
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
constexpr int kSlice = 32;   // value dims of a CTA with [dv, dk] states
constexpr int kWide = 64;    // and with [dk, dv] states
// CTAs of an SM that the registers leave room for: of [dk, dv] states by the
// state's size (four of d = 128 spill: 512 x 16 states 184 us), of [dv, dk] ones by the query
// heads of the first round.
template <int D>
constexpr int kStepPerSm = D == 128 ? 3 : 4;
template <typename T>
constexpr int kVfirstPerSm[5] = {0, sizeof(T) == 2 ? 5 : 4, sizeof(T) == 2 ? 5 : 4, 0, sizeof(T) == 2 ? 4 : 3};
// Rows of a CTA with [dk, dv] and [dv, dk] states, at most.  Drafted
// tokens leave most rows nothing to do: with one row each, 14000 CTAs come and
// go for 3000 that work (40 us instead of 36; 256 sequences of 1 to 8 tokens 238 instead of 194, but
// 512 of one token 156 instead of 159).  [dk, dv] states: with one row the 256 sequences 210
// us instead of 192 and 512 of one token 161 instead of 159; with four the per-dim case above 45 instead of 43.
constexpr int kMaxRows[2] = {2, 4};

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
        if (j >= last) return n;   // n itself among them
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

// For each of R rows, from `row` on, and their slots (negative: a row that does not count): the
// last row of the slot, or kEarlier where a row before it has the slot, which that one then takes
// along.  The whole block searches, kScan slots of a thread at first.
constexpr int kEarlier = 0x7fffffff;
constexpr int kScan = 4, kMore = 12;
__device__ __forceinline__ void first_slots(const int32_t *slots, int n, int (&s)[kScan]) {
#pragma unroll
    for (int u = 0; u < kScan; u++) {
        const int j = u * kThreads + threadIdx.x;
        s[u] = j < n ? slots[j] : -1;
    }
}
template <int R>
struct alignas(4 * R) Lasts {
    int x[R];
};
template <int R>
struct Search {
    int slot[R], last[R], row;

    __device__ __forceinline__ void run(const int32_t *slots, int n, const int (&s)[kScan], Lasts<R> (*sh)[kWarps]) {
#pragma unroll
        for (int r = 0; r < R; r++) last[r] = row + r;
#pragma unroll
        for (int r = 1; r < R; r++)
#pragma unroll
            for (int e = 0; e < r; e++)
                if (slot[e] == slot[r]) last[r] = kEarlier;
#pragma unroll
        for (int u = 0; u < kScan; u++) look(u * kThreads + threadIdx.x, s[u]);
        // long batches: with tokens of few sequences in turn most rows are known to be kEarlier by now
        if (n <= kScan * kThreads || join(sh[0])) return;
        // a dozen on their way at once: up to 2048 rows cost one more latency (256 sequences of 8 tokens next to one
        // another 207 -> 200 us)
        for (int j = kScan * kThreads + threadIdx.x; j < n; j += kMore * kThreads) {
            int x[kMore];
#pragma unroll
            for (int u = 0; u < kMore; u++) x[u] = j + u * kThreads < n ? slots[j + u * kThreads] : -1;
#pragma unroll
            for (int u = 0; u < kMore; u++) look(j + u * kThreads, x[u]);
        }
    }
    // What the warps found; true where no row is left that counts and may be the first of its slot.
    __device__ __forceinline__ bool join(Lasts<R> *sh) {
        Lasts<R> own;
#pragma unroll
        for (int r = 0; r < R; r++) own.x[r] = __reduce_max_sync(0xffffffffu, last[r]);
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = own;
        __syncthreads();
        bool done = true;
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            const Lasts<R> v = sh[w];
#pragma unroll
            for (int r = 0; r < R; r++) last[r] = max(last[r], v.x[r]);
        }
#pragma unroll
        for (int r = 0; r < R; r++) done = done && (slot[r] < 0 || last[r] == kEarlier);
        return done;
    }

  private:
    __device__ __forceinline__ void look(int j, int s) {   // row j has slot s; the rows themselves have been compared
        const int what = j < row ? kEarlier : j;
#pragma unroll
        for (int r = 0; r < R; r++)
            if (s == slot[r]) last[r] = max(last[r], what);
    }
};

struct Params {
    const void *q, *k, *v, *beta;
    const float *g;
    const float *state;
    float *state_out;
    const int32_t *slots;
    void *o;
    int n, num_slots, H, G;
    float scale;
    int rows;   // of a CTA
};

// The rows of a CTA that are the first of their slot, which take its other rows along (bit i: row `row0` + i),
// and those that another CTA's row takes along and that the row before does not tell of (bit 16 + i).
// `own` gets the rows' slots, sh[1] the slots' last rows.  The whole block calls it, before a state is
// read: a row that is taken along must cost no state's bytes, and in place the other CTA may be writing it.
// All rows of a CTA in one search, the first slots on their way with the rows' own: 512 x 16 states take as
// long as with the search behind the states' loads (158 us), which took 495 us for 256 sequences of 8 tokens in turn
// (329 now) and 309 for 32 of 64 (214); the drafted tokens above 34 (35).  What comes back is the same in every lane and
// the compiler has to know (a ballot): else the tokens' steps take more registers.
template <int R>
__device__ __forceinline__ uint32_t first_rows(const Params &p, int row0, int *own, Lasts<R> (*sh)[kWarps]) {
    const int lane = threadIdx.x & 31, row = row0 + lane;
    const bool there = lane < p.rows && row < p.n;
    uint32_t may = __ballot_sync(0xffffffffu, there);
    Search<R> f;
    f.row = row0;
#pragma unroll
    for (int r = 0; r < R; r++) {
        f.slot[r] = -1 - r;
        f.last[r] = row0 + r;
    }
    if (p.slots) {
        int s[kScan];
        first_slots(p.slots, p.n, s);
        const int slot = there ? p.slots[row] : -1, before = there && row ? p.slots[row - 1] : -1;
        // most rows that do not count are told by the row before
        may = __ballot_sync(0xffffffffu, slot >= 0 && slot < p.num_slots && slot != before);
        if (!may) return 0;
        if (p.n > 1) {
#pragma unroll
            for (int r = 0; r < R; r++) {
                const int x = __shfl_sync(0xffffffffu, slot, r);
                f.slot[r] = may >> r & 1 ? x : -1 - r;
            }
            f.run(p.slots, p.n, s, sh);
        }
        if (threadIdx.x < R) own[lane] = slot;
    }
    f.join(sh[1]);
    uint32_t others = 0;
#pragma unroll
    for (int r = 0; r < R; r++)
        if (may >> r & 1 && f.last[r] == kEarlier) others |= 1u << r;
    return __ballot_sync(0xffffffffu, ((may & ~others) | others << 16) >> lane & 1);
}

// What head x % H of row x / H reads, into the L2: the CTA that takes the row along finds it there (4
// sequences of 256 tokens in turn 361 -> 270 us).
template <typename T, int D, bool KDA>
__device__ __forceinline__ void fetch_token(const Params &p, int64_t x) {
    constexpr int per = 128 / (int)sizeof(T);   // values of a line
    auto warm = [](const void *a) { asm volatile("prefetch.global.L2 [%0];" ::"l"(a)); };
    for (int i = threadIdx.x * per; i < p.G * D; i += kThreads * per) warm((const T *)p.q + x * p.G * D + i);
    if ((int)threadIdx.x < D / per) {
        warm((const T *)p.k + x * D + threadIdx.x * per);
        warm((const T *)p.v + x * D + threadIdx.x * per);
    }
    if (KDA && threadIdx.x < D / 32) warm(p.g + x * D + threadIdx.x * 32);
}

// Four columns of a row.
struct Quad {
    float2 x, y;
};
__device__ __forceinline__ Quad mul(float2 a, const Quad &b) { return Quad{mul2(a, b.x), mul2(a, b.y)}; }
__device__ __forceinline__ void fma(Quad &c, float2 a, const Quad &b) {
    c.x = fma2(a, b.x, c.x);
    c.y = fma2(a, b.y, c.y);
}

// Four neighbouring values as loaded.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
    float4 r;
    __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = r; }
    __device__ __forceinline__ Quad wide() const { return Quad{make_float2(r.x, r.y), make_float2(r.z, r.w)}; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint2 *>(p) = r; }
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
template <typename T, int D, bool KDA, int GP>
__global__ void __launch_bounds__(kThreads, kVfirstPerSm<T>[GP]) delta_step_vfirst_kernel(Params p) {
    constexpr int L = D / 4, PER = 32 / L;        // lanes of a value dim, value dims of one load
    constexpr int N = 8 / PER;                    // value dims of a thread
    __shared__ Lasts<kMaxRows[1]> shared_last[2][kWarps];
    __shared__ int own_slots[kMaxRows[1]];
    next_grid_may_start();
    previous_grid_done();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x / (D / kSlice);
    const int v0 = blockIdx.x % (D / kSlice) * kSlice + w * 8 + lane / L, k0 = lane % L * 4;   // value dims v0 + PER i
    const int own = lane % L / (L / N);           // the value dim whose sums end up here
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
    const int row0 = blockIdx.y * p.rows;
    const uint32_t found = first_rows<kMaxRows[1]>(p, row0, own_slots, shared_last);
    for (uint32_t others = blockIdx.x % (D / kSlice) ? 0 : found >> 16; others; others &= others - 1)
        fetch_token<T, D, KDA>(p, (int64_t)(row0 + __ffs(others) - 1) * p.H + h);
    for (uint32_t firsts = found & 0xffff; firsts; firsts &= firsts - 1) {
        const int at_bit = __ffs(firsts) - 1, row = row0 + at_bit, slot = p.slots ? own_slots[at_bit] : row;
        int last = row;
#pragma unroll
        for (int x = 0; x < kWarps; x++) last = max(last, shared_last[1][x].x[at_bit]);
        load(row);
        const int64_t so = (((int64_t)slot * p.H + h) * D + v0) * D + k0;
        Quad S[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float4 x = *reinterpret_cast<const float4 *>(p.state + so + PER * i * D);
            S[i] = Quad{make_float2(x.x, x.y), make_float2(x.z, x.w)};
        }
        Rows rows(p.slots, p.n, slot, row, last);
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
}

// [dk, dv] states: a warp holds 16 value dims of all key dims and needs no other
// warp.  A lane has four of the value dims and D / 8 neighbouring key dims, so
// that a load takes 64 bytes of each of 8 rows, and sums over the key dims go
// over the 8 lanes of the same value dims.  A token's k, q and gate factors
// come from the warp's own place in shared memory, each as a pair of the
// same value for packed arithmetic, the groups of key dims 16 bytes off each
// other's banks.
template <int D, bool KDA, int GP>
struct Token {
    static constexpr int N = D / 8, ROW = N + 2;
    alignas(16) float2 k[8 * ROW];
    alignas(16) float2 q[GP][8 * ROW];
    alignas(16) float2 a[KDA ? 8 * ROW : 2];
};
template <typename T, int D, bool KDA, int GP>
__global__ void __launch_bounds__(kThreads, kStepPerSm<D>) delta_step_kernel(Params p) {
    using Tok = Token<D, KDA, GP>;
    constexpr int N = Tok::N;                     // key dims of a lane
    __shared__ Lasts<kMaxRows[0]> shared_last[2][kWarps];
    __shared__ int own_slots[kMaxRows[0]];
    __shared__ Tok toks[kWarps];
    next_grid_may_start();
    previous_grid_done();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x / (D / kWide), v0 = blockIdx.x % (D / kWide) * kWide + w * 16 + (lane & 3) * 4;
    const int k0 = (lane >> 2) * N;               // key dims k0 + i
    const int own = lane >> 3 & 3;                // after spread(): the value dim of the four whose sums end up here
    const int d0 = lane * 4;                      // the dims that this lane fetches of k, q and the gate
    const bool fetches = d0 < D;
    Tok &t = toks[w];
    const int place = d0 + d0 / N * 2, mine = (lane >> 2) * Tok::ROW;
    // one token as loaded, fetched while the one before runs
    struct Raw {
        Raw4<T> k, q[GP], v;
        T beta;
        float4 a;
    } f;
    auto load = [&](int j) {
        const int64_t hk = (int64_t)j * p.H + h, hq = hk * p.G;
        if (fetches) {
            f.k.load((const T *)p.k + hk * D + d0);
#pragma unroll
            for (int g = 0; g < GP; g++) f.q[g].load((const T *)p.q + (hq + (g < p.G ? g : 0)) * D + d0);
            if (KDA) f.a = *reinterpret_cast<const float4 *>(p.g + hk * D + d0);
        }
        if (!KDA) f.a.x = p.g[hk];
        f.v.load((const T *)p.v + hk * D + v0);
        f.beta = ((const T *)p.beta)[hk];
    };
    auto lay = [&](float2 *to, const Quad &x) {   // each of the four twice
        if (!fetches) return;
        *reinterpret_cast<float4 *>(to + place) = make_float4(x.x.x, x.x.x, x.x.y, x.x.y);
        *reinterpret_cast<float4 *>(to + place + 2) = make_float4(x.y.x, x.y.x, x.y.y, x.y.y);
    };
    auto pair_at = [&](const float2 *from, int i) {   // two neighbouring key dims' pairs
        const float4 x = *reinterpret_cast<const float4 *>(from + mine + i);
        return Quad{make_float2(x.x, x.y), make_float2(x.z, x.w)};
    };
    // the four value dims' sums over the key dims: each lane ends up with that of dim `own`
    auto spread = [&](const Quad &x) {
        const bool up = lane & 16, odd = lane & 8;
        float2 keep = up ? x.y : x.x, give = up ? x.x : x.y;
        keep.x += __shfl_xor_sync(0xffffffffu, give.x, 16);
        keep.y += __shfl_xor_sync(0xffffffffu, give.y, 16);
        float r = (odd ? keep.y : keep.x) + __shfl_xor_sync(0xffffffffu, odd ? keep.x : keep.y, 8);
        return r + __shfl_xor_sync(0xffffffffu, r, 4);
    };
    const int row0 = blockIdx.y * p.rows;
    const uint32_t found = first_rows<kMaxRows[0]>(p, row0, own_slots, shared_last);
    for (uint32_t others = blockIdx.x % (D / kWide) ? 0 : found >> 16; others; others &= others - 1)
        fetch_token<T, D, KDA>(p, (int64_t)(row0 + __ffs(others) - 1) * p.H + h);
    for (uint32_t firsts = found & 0xffff; firsts; firsts &= firsts - 1) {
        const int at_bit = __ffs(firsts) - 1, row = row0 + at_bit, slot = p.slots ? own_slots[at_bit] : row;
        int last = row;
#pragma unroll
        for (int x = 0; x < kWarps; x++) last = max(last, shared_last[1][x].x[at_bit]);
        load(row);
        const int64_t so = (((int64_t)slot * p.H + h) * D + k0) * D + v0;
        Quad S[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float4 x = *reinterpret_cast<const float4 *>(p.state + so + i * D);
            S[i] = Quad{make_float2(x.x, x.y), make_float2(x.z, x.w)};
        }
        Rows rows(p.slots, p.n, slot, row, last);
        for (int j = row; j < p.n;) {
            const int64_t hq = ((int64_t)j * p.H + h) * p.G;
            T *out = (T *)p.o + hq * D + v0 + own;
            const Quad k = f.k.wide(), v = f.v.wide();
            float qk[GP];
            __syncwarp();   // the token before has been read
            lay(t.k, k);
#pragma unroll
            for (int g = 0; g < GP; g++) {
                const Quad q = f.q[g].wide();
                lay(t.q[g], q);
                qk[g] = fetches ? dot(q, k) : 0.f;
            }
            float2 a = both(0.f);
            if (KDA) lay(t.a, Quad{make_float2(expf(f.a.x), expf(f.a.y)), make_float2(expf(f.a.z), expf(f.a.w))});
            else a = both(expf(f.a.x));
            const float beta = (float)f.beta;
            const int next = rows.next(j);
            if (next < p.n) load(next);
            __syncwarp();
            Quad x{}, y[GP] = {};
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const Quad kk = pair_at(t.k, i);
                Quad aa{a, a};
                if (KDA) aa = pair_at(t.a, i);
                S[i] = mul(aa.x, S[i]);
                S[i + 1] = mul(aa.y, S[i + 1]);
                fma(x, kk.x, S[i]);
                fma(x, kk.y, S[i + 1]);
#pragma unroll
                for (int g = 0; g < GP; g++) {
                    const Quad qq = pair_at(t.q[g], i);
                    fma(y[g], qq.x, S[i]);
                    fma(y[g], qq.y, S[i + 1]);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2)
#pragma unroll
                for (int g = 0; g < GP; g++) qk[g] += __shfl_xor_sync(0xffffffffu, qk[g], o);
            const float2 vv = own & 2 ? v.y : v.x;
            const float d = beta * ((own & 1 ? vv.y : vv.x) - spread(x));
            const bool writes = (lane & 4) == 0;
#pragma unroll
            for (int g = 0; g < GP; g++) {
                const float o = p.scale * fmaf(qk[g], d, spread(y[g]));
                if (writes && g < p.G) put(out, g * D, o);
            }
            Quad dd;
            dd.x = make_float2(__shfl_sync(0xffffffffu, d, lane & 3), __shfl_sync(0xffffffffu, d, 8 + (lane & 3)));
            dd.y = make_float2(__shfl_sync(0xffffffffu, d, 16 + (lane & 3)), __shfl_sync(0xffffffffu, d, 24 + (lane & 3)));
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const Quad kk = pair_at(t.k, i);
                fma(S[i], kk.x, dd);
                fma(S[i + 1], kk.y, dd);
            }
            // the query heads behind the first GP read S' itself
            for (int g = GP; g < p.G; g++) {
                Raw4<T> r;
                if (fetches) r.load((const T *)p.q + (hq + g) * D + d0);
                __syncwarp();
                if (fetches) lay(t.q[0], r.wide());
                __syncwarp();
                Quad z{};
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const Quad qq = pair_at(t.q[0], i);
                    fma(z, qq.x, S[i]);
                    fma(z, qq.y, S[i + 1]);
                }
                const float o = p.scale * spread(z);
                if (writes) put(out, (int64_t)g * D, o);
            }
            j = next;
        }
#pragma unroll
        for (int i = 0; i < N; i++)
            *reinterpret_cast<float4 *>(p.state_out + so + i * D) = make_float4(S[i].x.x, S[i].x.y, S[i].y.x, S[i].y.y);
    }
}

// For each of R rows and their slots: the last row of the slot, or kEarlier where a row
// before it has the slot, which that one then takes along.  The whole block calls it; `sh`
// holds R ints per warp.
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

// The causal conv's tokens: y = act(b + sum_i w_i x_i) over a slot's W - 1 kept
// inputs (oldest first) and the row's own, which then is the newest one kept.  A
// thread owns four channels, whose weights stay in registers for the rows of its
// CTA; the loads of kConvRows rows are in flight at once.  512 rows of 6144 channels,
// W = 4, bf16: 11.5 us (eight channels a thread 14, rows of their own 54), of which
// the bytes take 7.3; the rest is a launch and 1.7 waves (80 registers: 912 CTAs at once of
// 1536), each waiting for slots, then windows.  More tokens of a slot come one after the other from HBM,
// some 0.8 us each next to one another and up to 1.7 in turn.
struct ConvParams {
    const void *x;
    const float *weight, *bias;
    const void *state;
    void *state_out;
    const int32_t *slots;
    void *y;
    int n, num_slots, channels, groups;   // groups of kConvRows rows of a CTA
};
template <typename T>
constexpr int kConvRows = sizeof(T) == 2 ? 4 : 2;

// as in the conv over sequences: the fast divide returns 0 once the denominator
// passes 2^126, where the exact quotient is below 1e-36
__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

// grid (channel blocks, blocks of rows)
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv1d_step_kernel(ConvParams p) {
    constexpr int NW = W > 1 ? W - 1 : 1, R = kConvRows<T>;
    __shared__ int shared_last[2][kWarps][R];
    next_grid_may_start();
    previous_grid_done();
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 4;
    const bool live = c < p.channels;   // the CTA stays whole for the rows' search
    const T *state = (const T *)p.state + c;
    const int64_t C = p.channels;
    Quad w[W], b{};
    if (live) {
        float f[4 * W];   // as they lie: the four channels' W weights
#pragma unroll
        for (int i = 0; i < 4 * W; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p.weight + (int64_t)c * W + i);
            f[i] = x.x;
            f[i + 1] = x.y;
            f[i + 2] = x.z;
            f[i + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < W; i++) w[i] = Quad{make_float2(f[i], f[W + i]), make_float2(f[2 * W + i], f[3 * W + i])};
        if (p.bias) {
            const float4 x = *reinterpret_cast<const float4 *>(p.bias + c);
            b = Quad{make_float2(x.x, x.y), make_float2(x.z, x.w)};
        }
    }
    // y of row j, and the window moved on
    auto token = [&](int j, Raw4<T> (&win)[NW], const Raw4<T> &x) {
        Quad z = b;
#pragma unroll
        for (int i = 0; i < W; i++) {
            const Quad t = i < W - 1 ? win[i < W - 1 ? i : 0].wide() : x.wide();
            z.x = fma2(w[i].x, t.x, z.x);
            z.y = fma2(w[i].y, t.y, z.y);
        }
        if (SILU) z = Quad{make_float2(silu(z.x.x), silu(z.x.y)), make_float2(silu(z.y.x), silu(z.y.y))};
        T *y = (T *)p.y + j * C + c;
        store2(y, z.x);
        store2(y + 2, z.y);
#pragma unroll
        for (int i = 0; i + 1 < W - 1; i++) win[i] = win[i + 1];
        if (W > 1) win[NW - 1] = x;
    };
    for (int i = 0; i < p.groups; i++) {
        const int row = (blockIdx.y * p.groups + i) * R;
        if (row >= p.n) break;
        int slot[R], last[R];
        bool used[R];
        Raw4<T> win[R][NW], x[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            last[r] = row + r;
            slot[r] = row + r >= p.n ? -1 : p.slots ? p.slots[row + r] : row + r;
            used[r] = slot[r] >= 0 && slot[r] < p.num_slots;
        }
#pragma unroll
        for (int r = 0; r < R; r++)
            if (live && used[r]) x[r].load((const T *)p.x + (row + r) * C + c);
        // the windows of the rows that take their slot's others along alone: in place another CTA may be
        // writing the others' (512 rows as above 11.4 us with the windows behind the search and 11.6 ahead of it, 2048 rows 39.5 and 38.4)
        if (p.slots) last_rows<R>(p.slots, p.n, slot, row, last, shared_last[i & 1]);
#pragma unroll
        for (int r = 0; r < R; r++) {
            used[r] = used[r] && last[r] != kEarlier;
            if (!live || !used[r]) continue;
#pragma unroll
            for (int u = 0; u < W - 1; u++) win[r][u].load(state + ((int64_t)slot[r] * (W - 1) + u) * C);
        }
#pragma unroll
        for (int r = 0; r < R; r++) {
            if (!used[r]) continue;
            if (live) token(row + r, win[r], x[r]);
            if (last[r] > row + r) {   // more tokens of the slot
                Rows rows(p.slots, p.n, slot[r], row + r, last[r]);
                for (int j = rows.next(row + r); j < p.n; j = rows.next(j)) {
                    if (!live) continue;
                    Raw4<T> more;
                    more.load((const T *)p.x + j * C + c);
                    token(j, win[r], more);
                }
            }
            if (live) {
#pragma unroll
                for (int u = 0; u < W - 1; u++)
                    win[r][u].store((T *)p.state_out + ((int64_t)slot[r] * (W - 1) + u) * C + c);
            }
        }
    }
}

template <typename T, int W>
int conv_w(ConvParams p, bool silu, int sms, void *stream) {
    constexpr int per = kThreads * 4, R = kConvRows<T>;
    const int blocks = (p.channels + per - 1) / per, groups = (p.n + R - 1) / R;
    // several groups of rows for a CTA, which reads the weights once for them, as long as there are CTAs for the GPU
    p.groups = (int)std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)groups * blocks / (8 * sms)));
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
int launch_g(Params p, bool vfirst, int sms, void *stream) {
    const int64_t slices = (int64_t)p.H * (D / (vfirst ? kSlice : kWide)), busy = 2 * sms * (vfirst ? kVfirstPerSm<T>[GP] : kStepPerSm<D>);
    p.rows = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRows[vfirst], p.n * slices / busy));
    const dim3 grid((unsigned)slices, (unsigned)((p.n + p.rows - 1) / p.rows));
    return launch_early(vfirst ? delta_step_vfirst_kernel<T, D, KDA, GP> : delta_step_kernel<T, D, KDA, GP>, grid, kThreads, 0, 1,
                        stream, p);
}

template <typename T, int D, bool KDA>
int launch(const Params &p, bool vfirst, int sms, void *stream) {
    if (p.G == 1) return launch_g<T, D, KDA, 1>(p, vfirst, sms, stream);
    if (p.G == 2) return launch_g<T, D, KDA, 2>(p, vfirst, sms, stream);
    return launch_g<T, D, KDA, 4>(p, vfirst, sms, stream);
}

template <typename T>
int launch_t(const cpdr_ctx *c, const Params &p, void *stream) {
    const bool kda = c->plan.gate_kind == CPDR_GATE_PER_DIM, vf = c->plan.vfirst;
    const int sms = device_sms(c->device);
    if (c->plan.dk == 128) return kda ? launch<T, 128, true>(p, vf, sms, stream) : launch<T, 128, false>(p, vf, sms, stream);
    return kda ? launch<T, 64, true>(p, vf, sms, stream) : launch<T, 64, false>(p, vf, sms, stream);
}

}  // namespace

int launch_delta_step(const cpdr_ctx *c, const void *q, const void *k, const void *v, const void *beta, const float *g,
                      const float *state, float *state_out, const int32_t *slots, int n, int num_slots, void *o,
                      void *stream) {
    if (n == 0) return 0;
    const auto &pl = c->plan;
    const Params p{q, k, v, beta, g, state, state_out, slots, o, n, num_slots, pl.H, pl.G, pl.scale, 1};
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
