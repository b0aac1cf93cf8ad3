// hc_fp8.cuh -- 8-bit numbers with a scale for each block of 128: E4M3 codes
// (1 sign, 4 exponent bits with bias 7, 3 mantissa bits, no infinity, 0x7F and
// 0xFF stand for NaN) and scales, UE8M0 bytes (2^(byte - 127)) or fp32.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace hc {

constexpr int kFp8Block = 128;  // values of a row, or rows and columns of a matrix, that share a scale

// The UE8M0 byte of a group whose largest magnitude is amax: the smallest power of
// two at or above amax / 448, from 2^-126 on.  448 = 1.75 * 2^8, so with amax =
// 1.f * 2^(b - 127) it is 2^(b - 135), or twice that where 1.f > 1.75.  (Infinite: 2^120,
// at which the code 448 stands for more than fp32 holds.)
__device__ __forceinline__ uint32_t fp8_scale_byte(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
    return (uint32_t)(b < 1 ? 1 : b);
}
// 2^(127 - byte), the exact reciprocal of the scale of a byte from 1 to 253
__device__ __forceinline__ float fp8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two values, already divided by their scale, as codes (a in the low byte): nearest,
// ties to even, at most 448 in magnitude; NaN stays NaN.
__device__ __forceinline__ uint32_t fp8_codes(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// A scale as a number: fp32, or a UE8M0 byte (255 stands for NaN).
__device__ __forceinline__ float fp8_scale_value(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}
struct Fp8Scales {
    const void *p;
    int f32;
    // as it lies in memory (so that what is loaded early need not be looked at early), and its value
    __device__ __forceinline__ uint32_t raw(int64_t i) const {
        return f32 ? __ldg(static_cast<const uint32_t *>(p) + i) : __ldg(static_cast<const uint8_t *>(p) + i);
    }
    __device__ __forceinline__ float value(uint32_t r) const { return f32 ? __uint_as_float(r) : fp8_scale_value(r); }
    __device__ __forceinline__ float at(int64_t i) const { return value(raw(i)); }
};

}  // namespace hc
