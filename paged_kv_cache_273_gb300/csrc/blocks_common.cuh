// Device-side helpers of the kernels that keep state per block: 8-bit float
// caches (append_blocks.cu, decode_blocks.cuh) and key bounds (append_blocks.cu,
// select.cu).
#pragma once

#include "device_common.cuh"

namespace pkv {
namespace dev {

// Two floats -> two e4m3 codes (round to nearest even, saturating), x in the
// low byte; and back, exactly.
__device__ __forceinline__ uint32_t f8_pack(float x, float y)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(y), "f"(x));
    return d;
}

__device__ __forceinline__ void f8_unpack(uint32_t codes, float &x, float &y)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    const float2 f = half2_to_float2(h);
    x = f.x;
    y = f.y;
}

// Four e4m3 codes -> two fp16 pairs (codes 0, 1 and 2, 3), exactly.
__device__ __forceinline__ void f8x4_to_half2(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2_f32(int e)
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The exponent of a block's scale (a power of two), held within the range the
// append writes, whatever an unwritten block's scale may be.
__device__ __forceinline__ int block_exponent(float scale)
{
    const int e = (int)((__float_as_uint(scale) >> 23) & 255u) - 127;
    return min(max(e, BLOCK_MIN_EXP), BLOCK_MAX_EXP);
}

// The least e in the range of block exponents with amax <= 127 * 2^e (127 =
// 1.984375 * 2^6; amax >= 0): int8 steps for values up to amax.
__device__ __forceinline__ int int8_exponent(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return min(max(e, BLOCK_MIN_EXP), BLOCK_MAX_EXP);
}

}  // namespace dev
}  // namespace pkv
