// Matrix product with bias, activation and residual in its epilogue,
//     y = act(x w^T + bias) + residual,
// and its gradients  dz = dy act'(z),  dx = dz w,  dw = dz^T x,
// dbias = sum over rows of dz.  Operands are bf16, or (forward) e4m3 with one
// scale per row of x and one per row of w; products are accumulated in fp32
// in tensor memory and rounded once, behind the epilogue (dz is rounded to
// bf16 before the two gradient products: it is an operand of the tensor
// cores there; dbias is summed from the unrounded values).
//
// All of them are one product D[p, q] = sum_r A[p, r] B[q, r], whose operands
// lie in memory either along r (K-major: x, w, and dz for dx) or along p or q
// (MN-major: w for dx, dz and x for dw); the tensor maps and descriptors
// differ, nothing is transposed or copied.
//
// Two kernels:
//  * wide_kernel, bound by the tensor cores: pairs of CTAs (cta_group::2) own
//    256 x 256 tiles.  Per 128 bytes of r each CTA fetches 128 rows of A and
//    128 of B, 32 KiB per 512 tensor-core cycles: half of what a single CTA
//    with a 128 x 256 tile would draw from the L2.  Six stages of TMA loads,
//    one issuing thread, two accumulators of 256 TMEM columns, so that eight
//    epilogue warps empty one while the other fills; outputs leave through
//    swizzled staging tiles by TMA, which also cuts what lies outside the
//    matrix.  bf16 32768 x 2048 x 6144: 417 us, 1.98 PFLOP/s (the library's
//    product 413); e4m3 255 us, 3.23 PFLOP/s, in short runs and 273 to 288 in
//    longer ones; tensor pipe 92% and 86% active.
//  * narrow_kernel, for few rows of x, bound by reading w: 128 rows of w (the
//    128 lanes) by 16 to 128 rows of x (the columns) per CTA, with r split
//    over a cluster of up to 8 CTAs, whose partial sums meet in distributed
//    shared memory in the order of the CTAs.  16 x 2048 x 6144: 7.0 us
//    in a chain of calls, 8.5 in a graph (25 MB
//    of w, 3.7 us at the measured copy rate; the library's product 6.3): 2 us
//    until the unit has fetched the tensors' maps and the first bytes are
//    there, 3 us until the last of w, 1.5 for the partial sums and the epilogue.
#include <cuda.h>
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

using namespace tc;

constexpr int kRBytes = 128;   // bytes of r in a stage: 64 bf16 or 128 e4m3

struct Epilogue {
    const float *bias;       // [q] or NULL
    const float *xs, *ws;    // scales of e4m3 rows, or NULL
    const __nv_bfloat16 *residual;   // [p, q] or NULL (wide_kernel has it as a tensor map)
    int act;                 // 0 none, 1 SiLU, 2 GELU
    int has_z;               // the value before the activation is an output too
};

struct Args {
    Epilogue e;
    int64_t P, Q;            // rows and columns of D
    int blocks;              // stages of r
    int tiles_p, tiles_q;    // wide_kernel: tiles, and how many of them stay whole
    int whole;
    __nv_bfloat16 *y, *z;    // narrow_kernel
    int32_t *status;
};

// ------------------------------------------------------------------ helpers
__device__ __forceinline__ uint32_t ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// True in one thread of the warp, always the same, which the compiler then
// knows to be one: by "lane == 0" it wraps every product and copy in a loop
// over the active threads, 152 cycles a product where the tensor cores need 128.
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// The shared-memory address of the same place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tile load {x, y}, completing on the barrier at cluster address `bar`.
template <int GROUP>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y) {
    if (GROUP == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%3, %4}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
            "[%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
            : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *m, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The stores of this thread have read their tiles.
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

template <int GROUP, bool E4M3>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (GROUP == 2 && !E4M3)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
    else if (GROUP == 2)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
    else if (!E4M3)
        mma_bf16(d, a, b, idesc, acc);
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// Arrives, when all products issued so far are done, on the barrier at this
// place in both CTAs of the pair.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// Instruction descriptor: fp32 accumulator; bf16 (format 1) or e4m3 (format 0) operands.
template <bool E4M3, bool A_MN, bool B_MN>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N) {
    return (1u << 4) | ((E4M3 ? 0u : 1u) << 7) | ((E4M3 ? 0u : 1u) << 10) | ((A_MN ? 1u : 0u) << 15) |
           ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// An operand's stage of 128 rows (or of `rows` rows, K-major) by 128 bytes of
// r, 128-byte swizzle.  K-major: rows of 128 bytes, a 32-byte step of r is 32
// bytes on.  MN-major: two columns of 64 rows by 64 r, 8 KiB apart, a step of
// 16 r is 2 KiB on.
template <bool MN>
__device__ __forceinline__ uint64_t stage_desc(uint32_t addr) {
    return MN ? sdesc(addr, 8192, 1024) : sdesc(addr, 16, 1024);
}
template <bool MN>
constexpr uint64_t kStep = MN ? 2048 >> 4 : 32 >> 4;
template <int GROUP, bool MN, bool E4M3>
__device__ __forceinline__ void load_stage(uint32_t dst, const CUtensorMap *m, uint32_t bar, int row, int block) {
    const int r = block * (E4M3 ? 128 : 64);
    if (MN) {
        tma_load<GROUP>(dst, m, bar, row, r);
        tma_load<GROUP>(dst + 8192, m, bar, row + 64, r);
    } else {
        tma_load<GROUP>(dst, m, bar, r, row);
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2E = 1.44269504088896341f;

// erfc(a / sqrt 2) / 2 for 0 <= a: exp(-a^2 / 2) times a polynomial in
// t = 1 / (1 + 0.2925 a), the form of Abramowitz and Stegun 7.1.26, whose own
// coefficients keep only the absolute error small (1% of the value at a = 8).
// These were fitted to both, by linear programming over 0 <= a <= 13.5: off by at
// most 6.4e-8, and by at most 6.4e-5 of the value.  Less than half of the code
// of erff, whose two branches made the epilogue longer than the products.
// `e` becomes exp(-a^2 / 2); past a = 13.2 it is zero.
constexpr float tail_coef(int i) {
    constexpr float k[6] = {0.11755388629936f, 0.10494834988949f, 0.16799651703861f, -0.07095000933451f, 0.26645483865784f,
                            -0.08600364625295f};
    return k[i];
}
__device__ __forceinline__ float upper_tail(float a, float &e) {
    const float t = rcp_fast(fmaf(0.2925f, a, 1.f));
    e = exp2_fast(-0.5f * kLog2E * a * a);
    float p = fmaf(t, tail_coef(5), tail_coef(4));
#pragma unroll
    for (int i = 3; i >= 0; i--) p = fmaf(t, p, tail_coef(i));
    return p * t * e;
}
// SiLU z sigmoid(z); the quotient is 0 once its denominator passes 2^126, where
// the exact one is below 1e-36.
__device__ __forceinline__ float silu(float z) { return z * rcp_fast(1.f + exp2_fast(-kLog2E * z)); }
// GELU z Phi(z) = max(z, 0) - |z| Phi(-|z|); past 40 the second term is zero.
__device__ __forceinline__ float gelu(float z) {
    float e, m;
    const float a = fminf(fabsf(z), 40.f);
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(z), "f"(0.f));
    return fmaf(-a, upper_tail(a, e), m);
}
// The same for two values.
__device__ __forceinline__ float2 gelu2(float2 z) {
    using namespace vio;
    const float2 a = make_float2(fminf(fabsf(z.x), 40.f), fminf(fabsf(z.y), 40.f));
    const float2 d = fma2(a, both(0.2925f), both(1.f));
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    const float2 x = mul2(mul2(a, both(-0.5f * kLog2E)), a);
    const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
    float2 p = fma2(t, both(tail_coef(5)), both(tail_coef(4)));
#pragma unroll
    for (int i = 3; i >= 0; i--) p = fma2(t, p, both(tail_coef(i)));
    float2 m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.x) : "f"(z.x), "f"(0.f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m.y) : "f"(z.y), "f"(0.f));
    return fma2(mul2(mul2(p, t), e), mul2(a, both(-1.f)), m);
}
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if (ACT == 1) {
        const float s = rcp_fast(1.f + exp2_fast(-kLog2E * z));
        return s * fmaf(z, 1.f - s, 1.f);
    }
    float e;
    const float h = upper_tail(fabsf(z), e);
    return fmaf(0.39894228040143268f * z, e, z > 0.f ? 1.f - h : h);
}

// ------------------------------------------------------------------ wide
constexpr int kTile = 256;               // rows and columns of a pair's tile
// With a residual, a staging tile for each piece of a warp's columns (the
// residual waits there) and a stage less; without, one tile and six stages
// (32768 x 2048 x 6144: 417 us, with five stages 434).
template <bool RES>
constexpr int kWideStages = RES ? 5 : 6;
constexpr int kHalfStage = 128 * kRBytes;
constexpr int kWideStage = 2 * kHalfStage;
constexpr int kEpiWarps = 8;
constexpr int kEpiCols = 256 / (kEpiWarps / 4);   // columns of a warp: two pieces of 64
static_assert(kEpiCols == 128, "two pieces");
constexpr int kPiece = 32 * 128;         // 32 rows of 64 bf16
template <bool RES>
constexpr int kStaging = RES ? 2 * kPiece : kPiece;   // a warp's
constexpr int kWideThreads = 32 * (kEpiWarps + 2);
template <bool RES>
constexpr size_t kWideBytes = (size_t)kWideStages<RES> * kWideStage + kEpiWarps * kStaging<RES> + 256 + 1024;
static_assert(kWideBytes<true> <= 227 * 1024 && kWideBytes<false> <= 227 * 1024,
              "a CTA's stages and staging fit its shared memory");

struct WideBars {
    uint64_t full[6], empty[6], acc_full[2], acc_empty[2], residual[kEpiWarps];
    Ctl ctl;
    uint32_t tmem;
};
static_assert(sizeof(WideBars) <= 256, "barriers");

// Waits until accumulator `acc` has its tile.  The products take as long as their
// blocks of r: the usual limit and 2000 cycles for each of them (they take up
// to 600; a sum over 6e8 rows lasts longer than the usual limit).
__device__ __noinline__ bool wait_products(WideBars *b, int acc, uint32_t phase, int blocks, int32_t *status) {
    const long long t0 = clock64(), limit = kWaitCycles + 2000LL * blocks;
    while (!mbar_try_wait_sleep(&b->acc_full[acc], phase, 200000u)) {
        if (b->ctl.abort) return false;
        if (clock64() - t0 > limit) {
            if (atomicCAS(status, 0, 1) == 0) {
                status[1] = 163;
                status[2] = (int32_t)blockIdx.x;
            }
            b->ctl.abort = 1;
            return false;
        }
    }
    return true;
}

// Tiles in groups of 8 rows of tiles, column by column inside a group, so
// that the tiles that run together share their operands in the L2.  (One B
// fetched for two pairs by multicast, in clusters of 4: 0.92 to 1.09 of these
// times, and 8 of the 152 SMs find no cluster: not worth a second kernel.)
__device__ __forceinline__ void tile_at(const Args &a, int i, int &tp, int &tq) {
    const int per = 8 * a.tiles_q, g = i / per, r = i - g * per;
    const int rows = min(8, a.tiles_p - 8 * g);
    tq = r / rows;
    tp = 8 * g + (r - tq * rows);
}
// The work of a pair: the first `whole` items are tiles, two each of those
// behind them are a tile's halves of 128 columns (whole_tiles).
struct Item {
    int p, q;      // first row and column
    bool half;
};
__device__ __forceinline__ int item_count(const Args &a) { return 2 * a.tiles_p * a.tiles_q - a.whole; }
__device__ __forceinline__ Item item_at(const Args &a, int i) {
    const int over = i - a.whole;
    const bool half = over >= 0;
    int tp, tq;
    tile_at(a, half ? a.whole + (over >> 1) : i, tp, tq);
    return Item{tp * kTile, tq * kTile + (half ? (over & 1) * (kTile / 2) : 0), half};
}

template <bool E4M3, bool A_MN, bool B_MN, bool RES>
__global__ void __launch_bounds__(kWideThreads, 1)
wide_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
            const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mz,
            const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap mbh, Args a) {
    constexpr int STAGES = kWideStages<RES>;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char *staging = base + STAGES * kWideStage;
    WideBars &b = *reinterpret_cast<WideBars *>(staging + kEpiWarps * kStaging<RES>);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, items = item_count(a);
    next_grid_may_start();
    if (threadIdx.x == 0) {
        b.ctl.abort = 0;
        for (int s = 0; s < STAGES; s++) {
            mbar_init(&b.full[s], 1);
            mbar_init(&b.empty[s], 1);
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(&b.acc_full[s], 1);
            mbar_init(&b.acc_empty[s], 2 * kEpiWarps);
        }
        for (int s = 0; s < kEpiWarps; s++) mbar_init(&b.residual[s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == kEpiWarps) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&b.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    if (w == kEpiWarps + 1 && lane == 0) {
        tma_prefetch_desc(&ma);
        tma_prefetch_desc(&mb);
        tma_prefetch_desc(&my);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    previous_grid_done();
    const uint32_t tmem = b.tmem;

    if (w == kEpiWarps) {
        // -------------------------------------------------------- loads
        if (elected()) {
            const uint32_t full0 = remote(&b.full[0], 0);
            int it = 0;
            for (int t = pair; t < items && !b.ctl.abort; t += pairs) {
                const Item job = item_at(a, t);
                const int p0 = job.p + (int)rank * 128, q0 = job.q + (int)rank * (job.half ? 64 : 128);
                for (int k = 0; k < a.blocks; k++, it++) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&b.empty[s], (uint32_t)(it / STAGES + 1) & 1u, &b.ctl, a.status, 160)) break;
                    if (rank == 0) mbar_arrive_expect_tx(&b.full[s], job.half ? kWideStage + kHalfStage : 2 * kWideStage);
                    const uint32_t dst = smem_u32(base + s * kWideStage), bar = full0 + 8u * s;
                    load_stage<2, A_MN, E4M3>(dst, &ma, bar, p0, k);
                    if (!job.half)
                        load_stage<2, B_MN, E4M3>(dst + kHalfStage, &mb, bar, q0, k);
                    else   // 64 rows: one box of either form
                        tma_load<2>(dst + kHalfStage, &mbh, bar, B_MN ? q0 : k * (E4M3 ? 128 : 64), B_MN ? k * 64 : q0);
                }
            }
        }
    } else if (w == kEpiWarps + 1) {
        // -------------------------------------------------------- products
        if (rank == 0 && elected()) {
            constexpr uint32_t id_whole = idesc_of<E4M3, A_MN, B_MN>(256, 256), id_half = idesc_of<E4M3, A_MN, B_MN>(256, 128);
            const uint64_t ad = stage_desc<A_MN>(smem_u32(base)), bd = stage_desc<B_MN>(smem_u32(base + kHalfStage));
            int it = 0, n = 0;
            for (int t = pair; t < items && !b.ctl.abort; t += pairs, n++) {
                const int acc = n & 1;
                const uint32_t id = t < a.whole ? id_whole : id_half;
                if (!mbar_wait(&b.acc_empty[acc], (uint32_t)((n >> 1) + 1) & 1u, &b.ctl, a.status, 161)) break;
                tc_fence_after();
                for (int k = 0; k < a.blocks; k++, it++) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&b.full[s], (uint32_t)(it / STAGES) & 1u, &b.ctl, a.status, 162)) break;
                    const uint64_t so = (uint64_t)(s * kWideStage) >> 4;
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        mma<2, E4M3>(tmem + acc * 256, ad + so + j * kStep<A_MN>, bd + so + j * kStep<B_MN>, id,
                                     (k | j) ? 1u : 0u);
                    commit_pair(&b.empty[s]);
                }
                commit_pair(&b.acc_full[acc]);
            }
        }
    } else {
        // -------------------------------------------------------- epilogue
        // warp w: TMEM lanes (rows) 32 (w % 4) .. + 31, columns 128 (w / 4) ..
        // + 127 in two pieces of 64 (of half a tile: 64 (w / 4) .. + 63).  The residual's pieces come into the
        // staging tiles by TMA while the products run (a lane owns a row, and 32
        // rows are 32 lines to a load instruction: fetched by loads they took
        // 3000 cycles of a tile), and y takes their place.
        // Where z is wanted too, a second pass over the piece writes it.
        const int quad = w & 3;
        unsigned char *mine = staging + w * kStaging<RES>;
        const uint32_t empty0 = remote(&b.acc_empty[0], 0);
        int n = 0, fetched = 0;
        for (int t = pair; t < items; t += pairs, n++) {
            const int acc = n & 1;
            const Item it = item_at(a, t);
            const int last = it.half ? 0 : 1, c0 = (w >> 2) * (it.half ? kEpiCols / 2 : kEpiCols);
            const int64_t p0 = (int64_t)it.p + rank * 128 + quad * 32, p = p0 + lane;
            const int64_t q0 = (int64_t)it.q + c0;
            const float xs = a.e.xs && p < a.P ? a.e.xs[p] : 1.f;
            const int pieces = p0 < a.P ? (q0 + 64 < a.Q ? 1 + last : q0 < a.Q ? 1 : 0) : 0;   // that hold any of D
            if (RES && pieces && elected()) {
                tma_store_wait();   // the staging tiles have been read
                const uint32_t bar = smem_u32(&b.residual[w]);
                mbar_arrive_expect_tx(&b.residual[w], pieces * kPiece);
                for (int i = 0; i < pieces; i++)
                    tma_load<1>(smem_u32(mine + i * kPiece), &mr, bar, (int)q0 + 64 * i, (int)p0);
            }
            __syncwarp();
            // scales and bias of 32 columns, the next ones' on their way while these are used
            float4 sc[8], bi[8];
            auto columns = [&](int64_t q) {
#pragma unroll
                for (int g = 0; g < 8; g++) {
                    const bool in = q + 4 * g < a.Q;   // Q % 8 == 0
                    sc[g] = bi[g] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (a.e.ws && in) sc[g] = *reinterpret_cast<const float4 *>(a.e.ws + q + 4 * g);
                    if (a.e.bias && in) bi[g] = *reinterpret_cast<const float4 *>(a.e.bias + q + 4 * g);
                }
            };
            columns(q0);
            {
                const uint32_t phase = (uint32_t)(n >> 1) & 1u;
                const bool ok = mbar_try_wait(&b.acc_full[acc], phase) || wait_products(&b, acc, phase, a.blocks, a.status);
                if (!__all_sync(0xffffffffu, ok)) break;
            }
            tc_fence_after();
            if (RES && pieces && !warp_wait_all(&b.residual[w], (uint32_t)(fetched++) & 1u, &b.ctl, a.status, 164)) break;
#pragma unroll 1
            for (int i = 0; i <= last; i++) {
                unsigned char *tile = RES ? mine + i * kPiece : mine;
#pragma unroll 1
                for (int pass = 0; pass <= a.e.has_z; pass++) {
                    if (!RES || pass) {
                        if (elected()) tma_store_wait();   // the staging tile has been read
                        __syncwarp();
                    }
                    if (pass) columns(q0 + 64 * i);
#pragma unroll
                    for (int ch = 0; ch < 2; ch++) {
                        float v[32];
                        tmem_ld32(tmem + acc * 256 + c0 + 64 * i + 32 * ch + ((uint32_t)(32 * quad) << 16), v);
                        tmem_ld_wait();
                        if (i == last && ch == 1 && pass == a.e.has_z) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_remote(empty0 + 8u * acc);
                        }
                        if (i >= pieces) continue;
                        if (a.e.ws) {
#pragma unroll
                            for (int g = 0; g < 8; g++) {
                                v[4 * g] *= xs * sc[g].x;
                                v[4 * g + 1] *= xs * sc[g].y;
                                v[4 * g + 2] *= xs * sc[g].z;
                                v[4 * g + 3] *= xs * sc[g].w;
                            }
                        }
#pragma unroll
                        for (int g = 0; g < 8; g++) {
                            v[4 * g] += bi[g].x;
                            v[4 * g + 1] += bi[g].y;
                            v[4 * g + 2] += bi[g].z;
                            v[4 * g + 3] += bi[g].w;
                        }
                        columns(q0 + 64 * i + 32 * ch + 32);
                        if (pass == 0) {
                            if (a.e.act == 1) {
#pragma unroll
                                for (int j = 0; j < 32; j++) v[j] = silu(v[j]);
                            } else if (a.e.act == 2) {
#pragma unroll
                                for (int j = 0; j < 32; j += 2) {
                                    const float2 u = gelu2(make_float2(v[j], v[j + 1]));
                                    v[j] = u.x;
                                    v[j + 1] = u.y;
                                }
                            }
                        }
#pragma unroll
                        for (int g = 0; g < 4; g++) {
                            float *u = &v[g * 8];
                            uint4 *at = reinterpret_cast<uint4 *>(tile + sw128(lane, ch * 4 + g));
                            if (RES && pass == 0) {
                                float r[8];
                                vio::widen16(*at, r);
#pragma unroll
                                for (int j = 0; j < 8; j++) u[j] += r[j];
                            }
                            *at = make_uint4(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]), pack_bf16(u[4], u[5]),
                                             pack_bf16(u[6], u[7]));
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (i < pieces && elected()) tma_store(pass ? &mz : &my, smem_u32(tile), (int)q0 + 64 * i, (int)p0);
                }
            }
        }
        if (elected()) tma_store_wait();
    }
    __syncwarp();
    // After a wait that gave up, copies of this CTA may still be on their way.
    if (b.ctl.abort)
        for (int i = 0; i < 1000; i++) __nanosleep(1000);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (w == kEpiWarps) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ------------------------------------------------------------------ narrow
constexpr int kNarrowThreads = 32 * 6;
constexpr int kMaxSplit = 8;
template <int QN>
constexpr int kNarrowStage = (128 + QN) * kRBytes;
// CTAs of an SM, and the stages that this leaves to each beside its sums.
template <int QN>
constexpr int kNarrowPerSm = QN <= 32 ? 2 : 1;
template <int QN>
constexpr int narrow_sums() {   // groups of 4 columns, rounded up to every split
    int most = 0;
    for (int s = 2; s <= kMaxSplit; s++) most = most > (QN / 4 + s - 1) / s * s ? most : (QN / 4 + s - 1) / s * s;
    return most * 128 * 16;
}
template <int QN>
constexpr int kNarrowSums = narrow_sums<QN>();
template <int QN>
constexpr int kNarrowStages = (228 * 1024 / kNarrowPerSm<QN> - 3 * 1024 - kNarrowSums<QN>) / kNarrowStage<QN>;
struct NarrowBars {
    uint64_t full[8], empty[8], done, summed;
    Ctl ctl;
    uint32_t tmem;
};
template <int QN>
constexpr size_t kNarrowBytes = (size_t)kNarrowStages<QN> * kNarrowStage<QN> + kNarrowSums<QN> + sizeof(NarrowBars) + 1024;
static_assert(kNarrowStages<16> <= 8 && kNarrowStages<64> <= 8 && kNarrowStages<128> >= 3, "stages and their barriers");
// A kernel that started early waits for the one before it with its TMEM
// allocated, and must not hold what a block of that one still asks for: a wide
// block (all 512 columns) never shares its SM with another, and two narrow
// ones together take 256 columns at most.
static_assert(kWideBytes<true> + kNarrowBytes<16> > 228 * 1024 && kWideBytes<false> + kNarrowBytes<16> > 228 * 1024 &&
                  kWideBytes<true> + kNarrowBytes<32> > 228 * 1024 && kWideBytes<false> + kNarrowBytes<32> > 228 * 1024,
              "no block is left without its TMEM columns");

// The sum of a group of 4 columns over the CTAs of a cluster, in their order.
template <int SPLIT>
__device__ __forceinline__ void add_group(const float4 *s, float (&d)[4]) {
    float4 u[SPLIT];
#pragma unroll
    for (int z = 0; z < SPLIT; z++) u[z] = s[z * 128];
#pragma unroll
    for (int z = 0; z < SPLIT; z++) {
        d[0] += u[z].x;
        d[1] += u[z].y;
        d[2] += u[z].z;
        d[3] += u[z].w;
    }
}

// D here is transposed: lanes are rows of w (q of y), columns rows of x (p of
// y).  grid: (split, tiles of 128 rows of w, tiles of QN rows of x), cluster (split, 1, 1)
template <int QN, bool E4M3, bool A_MN>
__global__ void __launch_bounds__(kNarrowThreads, kNarrowPerSm<QN>)
narrow_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, Args a) {
    constexpr int STAGES = kNarrowStages<QN>, STAGE = kNarrowStage<QN>;
    constexpr int COLS = QN < 32 ? 32 : QN;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    float4 *sums = reinterpret_cast<float4 *>(base + STAGES * STAGE);   // [this CTA's groups of 4 columns][split][128 rows]
    NarrowBars &b = *reinterpret_cast<NarrowBars *>(base + STAGES * STAGE + kNarrowSums<QN>);
    const int w = threadIdx.x >> 5;
    const int split = gridDim.x, rank = blockIdx.x;
    const int64_t q0 = (int64_t)blockIdx.y * 128, p0 = (int64_t)blockIdx.z * QN;
    const int k0 = (int)((int64_t)a.blocks * rank / split), n = (int)((int64_t)a.blocks * (rank + 1) / split) - k0;
    auto load = [&](int it) {
        const int s = it % STAGES;
        mbar_arrive_expect_tx(&b.full[s], STAGE);
        const uint32_t dst = smem_u32(base + s * STAGE), bar = smem_u32(&b.full[s]);
        load_stage<1, A_MN, E4M3>(dst, &mw, bar, (int)q0, k0 + it);
        load_stage<1, false, E4M3>(dst + 128 * kRBytes, &mx, bar, (int)p0, k0 + it);
    };
    next_grid_may_start();
    if (w == 4) {
        // the first loads do not wait for the rest to be set up
        if (elected()) {
            tma_prefetch_desc(&mw);
            tma_prefetch_desc(&mx);
            b.ctl.abort = 0;
            for (int s = 0; s < STAGES; s++) {
                mbar_init(&b.full[s], 1);
                mbar_init(&b.empty[s], 1);
            }
            mbar_init(&b.done, 1);
            mbar_init(&b.summed, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            previous_grid_done();
            for (int it = 0; it < min(n, STAGES); it++) load(it);
        }
    } else if (w == 5) {
        tmem_alloc(&b.tmem, COLS);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    previous_grid_done();
    // waited for before the sums go out: the CTAs of the cluster have all begun
    if (split > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const uint32_t tmem = b.tmem;
    bool ok = true;
    float v[QN], bias = 0.f, ws = 1.f;
    if (w < 4 && q0 + threadIdx.x < a.Q) {
        if (a.e.bias) bias = a.e.bias[q0 + threadIdx.x];
        if (a.e.ws) ws = a.e.ws[q0 + threadIdx.x];
    }
    if (w == 4) {
        if (elected()) {
            for (int it = STAGES; it < n; it++) {
                if (!mbar_wait(&b.empty[it % STAGES], (uint32_t)(it / STAGES + 1) & 1u, &b.ctl, a.status, 170)) break;
                load(it);
            }
        }
        __syncwarp();
    } else if (w == 5) {
        if (elected()) {
            constexpr uint32_t id = idesc_of<E4M3, A_MN, false>(128, QN);
            const uint64_t ad = stage_desc<A_MN>(smem_u32(base)), bd = stage_desc<false>(smem_u32(base + 128 * kRBytes));
            for (int it = 0; it < n; it++) {
                const int s = it % STAGES;
                if (!mbar_wait(&b.full[s], (uint32_t)(it / STAGES) & 1u, &b.ctl, a.status, 171)) break;
                const uint64_t so = (uint64_t)(s * STAGE) >> 4;
#pragma unroll
                for (int j = 0; j < 4; j++)
                    mma<1, E4M3>(tmem, ad + so + j * kStep<A_MN>, bd + so + j * kStep<false>, id, (it | j) ? 1u : 0u);
                mma_commit(&b.empty[s]);
            }
            mma_commit(&b.done);
        }
        __syncwarp();
    } else {
        ok = warp_wait_all(&b.done, 0, &b.ctl, a.status, 172);
        tc_fence_after();
        const uint32_t at = tmem + ((uint32_t)(32 * w) << 16);
#pragma unroll
        for (int i = 0; i < QN; i += 16) tmem_ld16(at + i, *reinterpret_cast<float(*)[16]>(&v[i]));
        tmem_ld_wait();
    }
    // after a wait that gave up, copies of this CTA may still be on their way
    if (b.ctl.abort)
        for (int i = 0; i < 1000; i++) __nanosleep(1000);
    const int row = threadIdx.x;   // of the 128 rows of w, threads 0 .. 127
    const int64_t q = q0 + row;
    // groups of 4 columns whose sums a CTA of the cluster takes
    const int per = (QN / 4 + split - 1) / split, g0 = per * rank, groups = min(per, QN / 4 - g0);
    const bool mine = w < 4 && q < a.Q && ok;
    if (split > 1) {
        // every partial sum goes to the CTA that adds its group, which counts
        // the bytes; no CTA leaves before all of its own have come
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (w < 4) {
            if (threadIdx.x == 0 && groups > 0) mbar_arrive_expect_tx(&b.summed, (uint32_t)(groups * split * 2048));
            int owner = 0, at = 0;
            uint32_t to = remote(sums + rank * 128 + row, 0), bar = remote(&b.summed, 0);
#pragma unroll
            for (int i = 0; i < QN; i += 4) {
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                                 to + (uint32_t)(at * split * 2048)),
                             "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3]), "r"(bar)
                             : "memory");
                if (++at == per) {
                    at = 0;
                    if (++owner < split) {
                        to = remote(sums + rank * 128 + row, owner);
                        bar = remote(&b.summed, owner);
                    }
                }
            }
            if (groups > 0) ok = warp_wait_all(&b.summed, 0, &b.ctl, a.status, 173) && ok;
        }
    }
    if (mine && ok) {
        // columns (rows of x) i .. i + M - 1: what the epilogue reads of them is
        // loaded for all at once
        auto out = [&](int i, auto &d) {
            constexpr int M = sizeof(d) / sizeof(float);
            const int64_t p = p0 + i, o = p * a.Q + q;
            const int n = (int)min((int64_t)M, a.P - p);
            __nv_bfloat16 r[M];
            float xs[M];
#pragma unroll
            for (int j = 0; j < M; j++) {
                r[j] = __nv_bfloat16(0.f);
                xs[j] = 1.f;
            }
            if (a.e.residual) {
#pragma unroll
                for (int j = 0; j < M; j++)
                    if (j < n) r[j] = a.e.residual[o + j * a.Q];
            }
            if (a.e.ws) {
#pragma unroll
                for (int j = 0; j < M; j++)
                    if (j < n) xs[j] = a.e.xs[p + j] * ws;
            }
            if (a.e.ws) {
#pragma unroll
                for (int j = 0; j < M; j++) d[j] *= xs[j];
            }
#pragma unroll
            for (int j = 0; j < M; j++) d[j] += bias;
            if (a.e.has_z) {
#pragma unroll
                for (int j = 0; j < M; j++)
                    if (j < n) a.z[o + j * a.Q] = __float2bfloat16_rn(d[j]);
            }
            if (a.e.act == 1) {
#pragma unroll
                for (int j = 0; j < M; j++) d[j] = silu(d[j]);
            } else if (a.e.act == 2) {
#pragma unroll
                for (int j = 0; j < M; j++) d[j] = gelu(d[j]);
            }
#pragma unroll
            for (int j = 0; j < M; j++)
                if (j < n) a.y[o + j * a.Q] = __float2bfloat16_rn(d[j] + __bfloat162float(r[j]));
        };
        if (split > 1) {
            // this CTA's groups, each summed in the order of the CTAs; four
            // groups at a time, which fill one another's latencies
            auto run = [&](auto s) {
                constexpr int S = decltype(s)::value;
                int i = 0;
                for (; i + 4 <= groups && p0 + 4 * (g0 + i) < a.P; i += 4) {
                    float d[16] = {};
#pragma unroll
                    for (int g = 0; g < 4; g++)
                        add_group<S>(sums + (i + g) * S * 128 + row, *reinterpret_cast<float(*)[4]>(&d[4 * g]));
                    out(4 * (g0 + i), d);
                }
                for (; i < groups && p0 + 4 * (g0 + i) < a.P; i++) {
                    float d[4] = {};
                    add_group<S>(sums + i * S * 128 + row, d);
                    out(4 * (g0 + i), d);
                }
            };
            switch (split) {
                case 2: run(std::integral_constant<int, 2>()); break;
                case 3: run(std::integral_constant<int, 3>()); break;
                case 4: run(std::integral_constant<int, 4>()); break;
                case 5: run(std::integral_constant<int, 5>()); break;
                case 6: run(std::integral_constant<int, 6>()); break;
                case 7: run(std::integral_constant<int, 7>()); break;
                default: run(std::integral_constant<int, 8>()); break;
            }
        } else {
#pragma unroll
            for (int i = 0; i < QN; i += 16)
                if (p0 + i < a.P) out(i, *reinterpret_cast<float(*)[16]>(&v[i]));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 5) tmem_dealloc(tmem, COLS);
}

// ------------------------------------------------------------------ dz
// dz = dy act'(z), rounded once, and its column sums over blocks of rows
// (from the unrounded values).  A block is 256 columns by `per` rows, a
// thread 8 columns of every 8th row, four rows' loads at a time.
template <int ACT>
__global__ void __launch_bounds__(256)
dz_kernel(const __nv_bfloat16 *dy, const __nv_bfloat16 *z, int64_t rows, int width, int per,
          __nv_bfloat16 *dz, float *part) {
    constexpr int AHEAD = 4;
    __shared__ float sh[8][256];
    next_grid_may_start();
    previous_grid_done();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int col = blockIdx.y * 256 + tx * 8;
    const int64_t r0 = (int64_t)blockIdx.x * per, r1 = min(rows, r0 + per);
    float sum[8] = {};
    if (col < width) {
        for (int64_t r = r0 + ty; r < r1; r += 8 * AHEAD) {
            uint4 dr[AHEAD], zr[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; j++) {
                dr[j] = zr[j] = make_uint4(0, 0, 0, 0);
                if (r + 8 * j < r1) {
                    dr[j] = vio::load16(dy + (r + 8 * j) * width + col);
                    if (ACT) zr[j] = vio::load16(z + (r + 8 * j) * width + col);
                }
            }
#pragma unroll
            for (int j = 0; j < AHEAD; j++) {
                if (r + 8 * j >= r1) break;
                float d[8];
                vio::widen16(dr[j], d);
                if (ACT) {
                    float u[8];
                    vio::widen16(zr[j], u);
#pragma unroll
                    for (int i = 0; i < 8; i++) d[i] *= act_grad<ACT>(u[i]);
                    vio::store16(dz + (r + 8 * j) * width + col, d);
                }
#pragma unroll
                for (int i = 0; i < 8; i++) sum[i] += d[i];
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < 8; i++) sh[ty][tx * 8 + i] = sum[i];
    __syncthreads();
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c < width) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) v += sh[i][threadIdx.x];
        part[(int64_t)blockIdx.x * width + c] = v;
    }
}

// ------------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<EncodeTiledFn>(ptr)
                   : nullptr;
    }();
    return fn;
}

// [rows, cols] row-major, box {bx, by}; what lies outside reads as zero and is not written.
bool encode(CUtensorMap *m, const void *p, bool e4m3, int64_t rows, int64_t cols, int bx, int by) {
    EncodeTiledFn fn = encoder();
    if (!fn) return false;
    const int es = e4m3 ? 1 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(cols * es)};
    cuuint32_t box[2] = {(cuuint32_t)bx, (cuuint32_t)by};
    cuuint32_t one[2] = {1, 1};
    return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One operand of a product: `rows` rows (of p or q) by `red` elements of r,
// stored [rows, red] (K-major) or [red, rows] (MN-major).
struct Operand {
    const void *p;
    int64_t rows, red;
    bool mn;
};
bool encode(CUtensorMap *m, const Operand &o, bool e4m3, int tile_rows) {
    return o.mn ? encode(m, o.p, e4m3, o.red, o.rows, 64, 64) : encode(m, o.p, e4m3, o.rows, o.red, e4m3 ? 128 : 64, tile_rows);
}


int64_t up(int64_t x, int64_t d) { return (x + d - 1) / d; }

// The last round's tiles are halved where that fits the pairs: a half's block
// of r takes 430 cycles (what its operands take to come) instead of 590, and
// half the epilogue (4096 x 4096 x 4096: 102 -> 93 us, e4m3 48 -> 44;
// 256 x 2048 x 6144: 16.2 -> 13.5, with GELU and a residual 21.1 -> 16.4).
int64_t whole_tiles(int64_t tiles, int pairs) {
    const int64_t rem = tiles % pairs;
    return 2 * rem <= pairs ? tiles - rem : tiles;
}

template <bool E4M3, bool A_MN, bool B_MN, bool RES = false>
int wide(const Operand &A, const Operand &B, Args a, void *y, void *z, int sms, cudaStream_t st) {
    CUtensorMap ma, mb, mbh, my, mz, mr;
    if (!encode(&ma, A, E4M3, 128) || !encode(&mb, B, E4M3, 128) || !encode(&mbh, B, E4M3, 64) || !encode(&my, y, false, a.P, a.Q, 64, 32) ||
        !encode(&mz, z ? z : y, false, a.P, a.Q, 64, 32) ||
        !encode(&mr, a.e.residual ? a.e.residual : y, false, a.P, a.Q, 64, 32))
        return (int)cudaErrorInvalidValue;
    a.tiles_p = (int)up(a.P, kTile);
    a.tiles_q = (int)up(a.Q, kTile);
    const int64_t tiles = (int64_t)a.tiles_p * a.tiles_q;
    if (tiles > (int64_t)0x1fffffff) return (int)cudaErrorInvalidValue;
    a.whole = (int)whole_tiles(tiles, sms / 2);
    const int pairs = (int)std::min<int64_t>(2 * tiles - a.whole, sms / 2);
    return launch_early(wide_kernel<E4M3, A_MN, B_MN, RES>, dim3(2 * pairs), kWideThreads, kWideBytes<RES>, 2, st, ma, mb, my, mz,
                        mr, mbh, a);
}

template <int QN, bool E4M3, bool A_MN>
int narrow(const Operand &W, const Operand &X, Args a, int split, cudaStream_t st) {
    CUtensorMap mw, mx;
    if (!encode(&mw, W, E4M3, 128) || !encode(&mx, X, E4M3, QN)) return (int)cudaErrorInvalidValue;
    const dim3 grid((unsigned)split, (unsigned)((a.Q + 127) / 128), (unsigned)((a.P + QN - 1) / QN));
    return launch_early(narrow_kernel<QN, E4M3, A_MN>, grid, kNarrowThreads, kNarrowBytes<QN>, split, st, mw, mx, a);
}

// Which kernel runs a product whose rows p are rows of x, by an estimate of
// its cycles from measured parts (64 x 2048 x 6144: 10.4 us narrow, 12.4 wide;
// 256 x 2048 x 6144: 38 us narrow with 128 rows of x a tile, 13.4 wide).
struct Choice {
    int qn = 0, split = 1;   // qn 0: wide_kernel
};
Choice choose(int64_t P, int64_t Q, int blocks, int sms) {
    Choice best;
    // tiles one after the other: 590 cycles for a block (512 are the products'),
    // 7000 for an epilogue that goes on meanwhile; the first load and the last
    // epilogue alone.  A round of halves: see whole_tiles.
    const int64_t wide_tiles = up(P, kTile) * up(Q, kTile), whole = whole_tiles(wide_tiles, sms / 2);
    double cost = (double)up(whole, sms / 2) * std::max(blocks * 590.0, 7000.0);
    cost += whole < wide_tiles ? std::max(blocks * 430.0, 3500.0) + 12000.0 : 10500.0;
    for (int qn = 16; qn <= 128; qn *= 2) {
        if (up(Q, 128) > 65535 || up(P, qn) > 65535) continue;
        const int64_t tiles = up(P, qn) * up(Q, 128);
        const int fit = qn <= 32 ? 2 : 1;
        const double block = std::max(2.0 * qn, (128 + qn) * kRBytes / 45.0);   // what an SM fetches in a cycle
        for (int split = 1; split <= kMaxSplit && split <= blocks; split++) {
            // a cluster of more than two finds no place on some of the last SMs
            const int64_t room = (int64_t)sms * fit * (split > 2 ? 15 : 16) / 16;
            const int64_t waves = up(tiles * split, room);
            const double together = waves > 1 ? fit : (double)up(tiles * split, sms);
            // a column's epilogue, or its partial sums to send and to add
            const double columns = split > 1 ? 1500.0 + 20.0 * qn * split : 200.0 * qn;
            const double c = waves * (up(blocks, split) * block * together + 7000.0 + columns);
            if (c < cost) {
                cost = c;
                best.qn = qn;
                best.split = split;
            }
        }
    }
    return best;
}

// D = X W^T for rows of x (K-major) and rows of w (K- or MN-major).
template <bool E4M3, bool W_MN>
int product(const Operand &X, const Operand &W, Args a, void *y, void *z, int sms, cudaStream_t st) {
    const Choice c = choose(a.P, a.Q, a.blocks, sms);
    a.y = (__nv_bfloat16 *)y;
    a.z = (__nv_bfloat16 *)z;
    switch (c.qn) {
        case 16: return narrow<16, E4M3, W_MN>(W, X, a, c.split, st);
        case 32: return narrow<32, E4M3, W_MN>(W, X, a, c.split, st);
        case 64: return narrow<64, E4M3, W_MN>(W, X, a, c.split, st);
        case 128: return narrow<128, E4M3, W_MN>(W, X, a, c.split, st);
        default: break;
    }
    if constexpr (!W_MN) {
        if (a.e.residual) return wide<E4M3, false, false, true>(X, W, a, y, z, sms, st);
    }
    return wide<E4M3, false, W_MN>(X, W, a, y, z, sms, st);
}

// Row blocks of dz_kernel: enough for eight blocks per SM, of 64 rows or more.
int dz_rows_per_block(int64_t rows, int width, int sms) {
    const int64_t want = std::max<int64_t>(1, (int64_t)sms * 8 / ((width + 255) / 256));
    return (int)std::max<int64_t>(64, (rows + want - 1) / want);
}

}  // namespace

int launch_linear_fwd(const cpdr_ctx *c, int64_t rows, int K, int N, const void *x, const void *w, const float *x_scale,
                      const float *w_scale, const float *bias, int act, const void *residual, void *z, void *y,
                      void *stream) {
    const bool e4m3 = x_scale != nullptr;
    Args a{};
    a.e = Epilogue{bias, x_scale, w_scale, (const __nv_bfloat16 *)residual, act, z ? 1 : 0};
    a.P = rows;
    a.Q = N;
    a.blocks = (K * (e4m3 ? 1 : 2) + kRBytes - 1) / kRBytes;
    a.status = c->dev.status;
    const Operand X{x, rows, K, false}, W{w, N, K, false};
    const int sms = device_sms(c->device);
    cudaStream_t st = (cudaStream_t)stream;
    return e4m3 ? product<true, false>(X, W, a, y, z, sms, st) : product<false, false>(X, W, a, y, z, sms, st);
}

void linear_plan(const cpdr_ctx *c, int64_t rows, int K, int N, bool e4m3, int32_t out[2]) {
    const Choice ch = choose(rows, N, (K * (e4m3 ? 1 : 2) + kRBytes - 1) / kRBytes, device_sms(c->device));
    out[0] = ch.qn;
    out[1] = ch.split;
}

size_t linear_dz_parts(const cpdr_ctx *c, int64_t rows, int N) {
    const int per = dz_rows_per_block(rows, N, device_sms(c->device));
    return (size_t)((rows + per - 1) / per);
}

int launch_linear_bwd(const cpdr_ctx *c, int64_t rows, int K, int N, const void *x, const void *w, const void *z,
                      const void *dy, int act, void *dx, void *dw, float *dbias, void *dz, float *part, void *stream) {
    const int sms = device_sms(c->device);
    cudaStream_t st = (cudaStream_t)stream;
    int rc = 0;
    if (act || dbias) {
        const int per = dz_rows_per_block(rows, N, sms);
        const int64_t parts = (rows + per - 1) / per;
        auto kernel = act == 0 ? dz_kernel<0> : act == 1 ? dz_kernel<1> : dz_kernel<2>;
        rc = launch_early(kernel, dim3((unsigned)parts, (unsigned)((N + 255) / 256)), 256, 0, 1, st, (const __nv_bfloat16 *)dy,
                          (const __nv_bfloat16 *)z, rows, N, per, (__nv_bfloat16 *)dz, dbias ? part : nullptr);
        if (rc) return rc;
        if (dbias) rc = launch_column_sums(part, (int)parts, N, dbias, stream);
        if (rc) return rc;
    }
    const void *g = act ? dz : dy;
    Args a{};
    a.status = c->dev.status;
    if (dx) {
        a.P = rows;
        a.Q = K;
        a.blocks = (N + 63) / 64;
        rc = product<false, true>(Operand{g, rows, N, false}, Operand{w, K, N, true}, a, dx, nullptr, sms, st);
        if (rc) return rc;
    }
    if (dw) {
        a.P = N;
        a.Q = K;
        a.blocks = (int)((rows + 63) / 64);
        rc = wide<false, true, true>(Operand{g, N, rows, true}, Operand{x, K, rows, true}, a, dw, nullptr, sms, st);
    }
    return rc;
}

}  // namespace cpdr
