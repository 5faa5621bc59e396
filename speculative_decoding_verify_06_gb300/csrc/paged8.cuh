// paged8.cuh -- the 8-bit page format shared by the paged-cache kernels that hold one.
//
// A page holds page_size positions (a multiple of 16) of every kv head as units of 16 positions,
// [page][kv head][page_size / 16][4112 bytes]:
//   bytes    0..2047  K codes [16 positions][128 B]: the 16 bytes of dims 16c .. 16c + 15 at place c ^ (position % 8), so that
//                     a unit copied to shared memory is a K-major operand with the 128-byte swizzle as it lies
//   bytes 2048..4095  V codes [128 dims][16 positions]
//   bytes 4096..4103  scales of the keys and of the values, fp32; 4104..4111: unused
// A code is an e4m3 float (largest 448); its value is code * scale.  Scales are powers of two, so that changing
// one changes no code but those among e4m3's subnormals.
#pragma once

#include "paged.cuh"

namespace svd {

constexpr int kP8UnitBytes = SVD_PAGED8_UNIT_BYTES;
constexpr int kP8VCodes = 2048;
constexpr int kP8Scales = 4096;
constexpr int kP8ExpLo = -64, kP8ExpHi = 7;  // of the scales
constexpr float kP8MaxAbs = 57344.f;         // 448 * 2^7: magnitudes end here

__device__ __forceinline__ float p8_pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
// The exponent of a stored scale (0 in pages never written).
__device__ __forceinline__ int p8_exponent(float scale) {
    return min(max((int)((__float_as_uint(scale) >> 23) & 255u) - 127, kP8ExpLo), kP8ExpHi);
}
// The smallest e with 448 * 2^e >= top (448 = 1.75 * 2^8), for finite top >= 0, not limited yet.
__device__ __forceinline__ int p8_need(float top) {
    const uint32_t u = __float_as_uint(top);
    return (int)(u >> 23) - 127 - ((u & 0x7FFFFFu) > 0x600000u ? 7 : 8);
}
// Two floats to codes (a in the low byte), to nearest even, and back.
__device__ __forceinline__ uint32_t p8_encode2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t p8_decode2(uint32_t codes) {  // a pair of fp16, exact
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}
__device__ __forceinline__ float2 p8_floats2(uint32_t codes) {
    const uint32_t h = p8_decode2(codes);
    return __half22float2(reinterpret_cast<const __half2 &>(h));
}

}  // namespace svd
