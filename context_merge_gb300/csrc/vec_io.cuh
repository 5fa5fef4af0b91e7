// Element access shared by the layer-step kernels: pairs of neighbouring
// channels and 16-byte vectors of fp32 or bf16, widened to fp32 where used.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace cpdr {
namespace vio {

// Two values in one instruction (round to nearest, as the scalar forms).
__device__ __forceinline__ uint64_t pair(float2 v) { return *reinterpret_cast<uint64_t *>(&v); }
__device__ __forceinline__ float2 unpair(uint64_t r) { return *reinterpret_cast<float2 *>(&r); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
    return unpair(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
    return unpair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
    return unpair(r);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Two neighbouring channels as loaded.
template <typename T>
struct Raw2;
template <>
struct Raw2<float> {
    float2 a;
};
template <>
struct Raw2<__nv_bfloat16> {
    uint32_t a;
};

__device__ __forceinline__ Raw2<float> load2(const float *p) {
    return Raw2<float>{*reinterpret_cast<const float2 *>(p)};
}
__device__ __forceinline__ Raw2<__nv_bfloat16> load2(const __nv_bfloat16 *p) {
    return Raw2<__nv_bfloat16>{*reinterpret_cast<const uint32_t *>(p)};
}
__device__ __forceinline__ float2 widen(const Raw2<float> &r) { return r.a; }
__device__ __forceinline__ float2 widen(const Raw2<__nv_bfloat16> &r) {
    // a bf16 is the upper half of the fp32 of the same value
    return make_float2(__uint_as_float(r.a << 16), __uint_as_float(r.a & 0xffff0000u));
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// 16 bytes of a row: 4 fp32 or 8 bf16.
template <typename T>
constexpr int kVecOf = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ uint4 load16(const T *p) {
    return *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void widen16(const uint4 &r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void widen16(const uint4 &r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store16(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&v)[8]) {
    uint4 r;
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; i++) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    r.x = *reinterpret_cast<uint32_t *>(&h[0]);
    r.y = *reinterpret_cast<uint32_t *>(&h[1]);
    r.z = *reinterpret_cast<uint32_t *>(&h[2]);
    r.w = *reinterpret_cast<uint32_t *>(&h[3]);
    *reinterpret_cast<uint4 *>(p) = r;
}

}  // namespace vio
}  // namespace cpdr
