// Scalar pieces that the attention kernels share.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace moe {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two e4m3 values, the lower or upper two bytes of v, as an fp16 pair, exact
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t v) {
    uint32_t d;
    asm("{.reg .b16 h, l; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t v) {
    uint32_t d;
    asm("{.reg .b16 h, l; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(d) : "r"(v));
    return d;
}
// x * y + z, x * y and x + y of both halves
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 d;
    asm("{.reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
        " fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 d;
    asm("{.reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 d;
    asm("{.reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}
// two numbers as bf16, the first in the lower half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// tanh z, off by 8 units of 2^-24 relative to itself: up to 1/2 by an odd polynomial, fitted
// to the least relative error there (1.5e-8), and where PAST, past it, by 1 - 2 / (exp(2 z) +
// 1), whose error of 2^-22 would be the larger the nearer to zero.
constexpr float kTanh3 = -0.333331439f, kTanh5 = 0.13325879f, kTanh7 = -0.0530454943f, kTanh9 = 0.0172414916f;
template <bool PAST>
__device__ __forceinline__ float tanh_of(float z) {
    const float u = z * z;
    const float r = z * fmaf(fmaf(fmaf(fmaf(kTanh9, u, kTanh7), u, kTanh5), u, kTanh3), u, 1.f);
    if (!PAST || !(fabsf(z) > 0.5f)) return r;
    return 1.f - 2.f * rcp(ex2(z * (2.f * kLog2e)) + 1.f);
}

}  // namespace moe
