// Scalar pieces that the attention kernels share.
#pragma once

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
// tanh z, off by 8 units of 2^-24 relative to itself: up to 1/2 by an odd polynomial, fitted
// to the least relative error there (1.5e-8), and where PAST, past it, by 1 - 2 / (exp(2 z) +
// 1), whose error of 2^-22 would be the larger the nearer to zero.
template <bool PAST>
__device__ __forceinline__ float tanh_of(float z) {
    const float u = z * z;
    const float r = z * fmaf(fmaf(fmaf(fmaf(0.0172414916f, u, -0.0530454943f), u, 0.13325879f), u, -0.333331439f), u, 1.f);
    if (!PAST || !(fabsf(z) > 0.5f)) return r;
    return 1.f - 2.f * rcp(ex2(z * (2.f * kLog2e)) + 1.f);
}

}  // namespace moe
