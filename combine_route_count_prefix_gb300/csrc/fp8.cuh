// fp8.cuh -- block-scaled e4m3: the quantisation of 128 columns shared by the
// norm and the fp8 FFN, and the conversions.
#pragma once
#include <cuda_fp8.h>
#include <stdint.h>

namespace moe {

constexpr int kFp8Block = 128;               // columns per scale
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 7.8886090522101181e-31f;   // 2^-100: 448 / it is finite

// Two floats -> two e4m3 codes (lo in the low byte), round to nearest even,
// saturating; NaN -> NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// 448 / a within two units in the last place, for a >= 2^-100.  The reciprocal
// is taken of a / 512, so that no finite a makes it a denormal.
__device__ __forceinline__ float inverse_scale(float a) {
    return __frcp_rn(a * 0x1p-9f) * (kE4m3Max * 0x1p-9f);
}
// Scale a / 448 and its inverse for a block whose largest magnitude is amax.
// (Two IEEE divisions per thread were half of the norm's instructions.)
__device__ __forceinline__ void block_scale(float amax, float &s, float &inv) {
    const float a = fmaxf(amax, kAmaxFloor);
    s = a * (1.0f / kE4m3Max);
    inv = inverse_scale(a);
}

// silu(a) * b, with the hardware's approximate exponential and reciprocal
// (relative error about 1e-7 + 1e-7 |a|, before a rounding to e4m3 at 6e-2):
// with expf and a division it was twice the instructions.
__device__ __forceinline__ float swiglu(float a, float b) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return a * r * b;
}

}  // namespace moe
