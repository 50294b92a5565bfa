// fp8.cuh -- e4m3 conversions and the 128-column block scale shared by the 8-bit kernels.
//
// A block of 128 values y is held as q = e4m3(y / scale) with one fp32 scale
//   scale = max(max|y| / 448, 2^-126),
// 448 being the largest e4m3 number. The floor keeps the scale of an all-zero (or tiny) block
// a normal number, so that q = 0 / scale = 0 needs no branch. The conversion rounds to nearest
// even (half a step: 2^-4 relative, 2^-10 * scale absolute below 2^-6 * scale) and saturates;
// NaN stays NaN.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace vit {

constexpr int kFp8Block = 128;   // columns (and, for weights, rows) that share one scale

// The quotient as a product with the rounded 1 / 448, at most one unit in the last place off, and
// the codes from the hardware reciprocal of the scale, likewise: IEEE division and reciprocal
// cost the HBM-bound kernels a third of their time (norm of 16400 x 1280 to e4m3: 37.6 us).
__device__ __forceinline__ float fp8_block_scale(float amax) {
    return fmaxf(amax * (1.f / 448.f), 1.17549435e-38f);
}
// 1 / scale; scales lie between 2^-126 and 2^120, or are infinite.
__device__ __forceinline__ float fp8_inverse(float scale) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
    return r;
}

// Two floats as two e4m3 codes, a in the low byte.
__device__ __forceinline__ uint32_t fp8_pack2(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    return fp8_pack2(a, b) | (fp8_pack2(c, d) << 16);
}
__device__ __forceinline__ uint8_t fp8_pack1(float a) {
    return (uint8_t)__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3);
}

// The exact values of e4m3 codes (each is an fp16 number).
__device__ __forceinline__ float fp8_value(uint8_t q) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)q, __NV_E4M3)));
}

}  // namespace vit
