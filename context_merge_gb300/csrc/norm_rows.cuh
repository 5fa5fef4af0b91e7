// Rows in the registers of a group of threads, shared by the norms: the
// groups and vectors for each width, and the 8-bit output.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "vec_io.cuh"

namespace cpdr {
namespace norm {

using vio::kVecOf;

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// V values times `inv` in e4m3, at d.
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t *d, const float (&s)[V], float inv) {
    uint32_t q[V / 4];
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[j] * inv, s[j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[j + 2] * inv, s[j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        q[j / 4] = lo | hi << 16;
    }
    if (V == 8)
        *reinterpret_cast<uint2 *>(d) = make_uint2(q[0], q[V / 4 - 1]);
    else
        *reinterpret_cast<uint32_t *>(d) = q[0];
}

template <int TPR>
constexpr int kBlock = TPR < 256 ? 256 : TPR;

template <int TPR, int NV, typename F>
int with(F f) {
    return f(std::integral_constant<int, TPR>(), std::integral_constant<int, NV>());
}

// Threads per row, and 16-byte vectors for each of them: groups of up to 256
// threads with one or two vectors, three where two would leave a quarter of
// the threads idle or more (bf16 rows of 264, forward 6.1 -> 7.0 TB/s and
// backward 3.3 -> 5.1).  Wider rows are each norm's own.
template <typename T, typename F>
int narrow_row(int vecs, F f) {
    if (vecs <= 1) return with<1, 1>(f);
    if (vecs <= 2) return with<2, 1>(f);
    if (vecs <= 4) return with<4, 1>(f);
    if (vecs <= 8) return with<8, 1>(f);
    if (vecs <= 12) return with<4, 3>(f);
    if (vecs <= 16) return with<16, 1>(f);
    if (vecs <= 24) return with<8, 3>(f);
    if (vecs <= 32) return with<32, 1>(f);
    if (vecs <= 48) return with<16, 3>(f);
    if (vecs <= 64) return with<32, 2>(f);
    if (vecs <= 96) return with<32, 3>(f);
    if (vecs <= 128) return with<64, 2>(f);
    if (vecs <= 192) return with<64, 3>(f);
    if (vecs <= 256) return with<128, 2>(f);
    if (vecs <= 384) return with<128, 3>(f);
    if (vecs <= 512) return with<256, 2>(f);
    return with<256, 3>(f);
}

}  // namespace norm
}  // namespace cpdr
