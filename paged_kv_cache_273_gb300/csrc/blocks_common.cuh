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

// The least e >= BLOCK_MIN_EXP with amax <= 448 * 2^e, the largest e4m3 value
// being 448 = 1.75 * 2^8 (amax finite, >= 0).
__device__ __forceinline__ int code_exponent(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, BLOCK_MIN_EXP), BLOCK_MAX_EXP);
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, m));
    return x;
}

// For every run that starts at a token of [t0, t0 + C) (C <= 32), in order:
// f(first token, block, first offset in the block, rows).  All lanes call f
// together.  `report`: record slots beyond the cache.
template <typename F>
__device__ __forceinline__ void for_runs(const int32_t *slots, int64_t t0, int C, int64_t T,
                                         int bs, int64_t num_slots, bool report,
                                         unsigned int *err, F f)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = t0 + lane;
    const int s = lane < C && t < T ? slots[t] : -1;
    int before = __shfl_up_sync(FULL_MASK, s, 1);
    if (lane == 0)
        before = t0 > 0 ? slots[t0 - 1] : -1;
    if (report && s >= 0 && (int64_t)s >= num_slots)
        atomicOr(err, PKV_EBIT_SLOT);
    const bool starts = s >= 0 && (int64_t)s < num_slots &&
                        (before != s - 1 || (s & (bs - 1)) == 0);
    unsigned todo = __ballot_sync(FULL_MASK, starts);
    while (todo) {
        const int i = __ffs(todo) - 1;
        todo &= todo - 1;
        const int slot = __shfl_sync(FULL_MASK, s, i);
        const int off = slot & (bs - 1);
        int n = 1;                                   // rows of the run
        for (;;) {
            const int64_t tn = t0 + i + n + lane;
            const bool more = off + n + lane < bs && tn < T && slots[tn] == slot + n + lane;
            const unsigned gap = ~__ballot_sync(FULL_MASK, more);
            if (gap) {
                n += __ffs(gap) - 1;
                break;
            }
            n += 32;
        }
        f(t0 + i, slot / bs, off, n);
    }
}

// A block's first n 16-byte pieces of e4m3 codes by 2^down (<= 0), a piece a lane of
// the warp: the rows that it holds when its exponent grows.
__device__ __forceinline__ void rescale_rows(uint8_t *rows, int n, int down)
{
    const float f = pow2_f32(max(down, -126));
    uint4 *p = reinterpret_cast<uint4 *>(rows);
    for (int i = threadIdx.x & 31; i < n; i += 32) {
        const uint4 old = p[i];
        uint32_t v[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float y[4];
            f8_unpack(v[u] & 0xffffu, y[0], y[1]);
            f8_unpack(v[u] >> 16, y[2], y[3]);
            v[u] = f8_pack(y[0] * f, y[1] * f) | f8_pack(y[2] * f, y[3] * f) << 16;
        }
        p[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

}  // namespace dev
}  // namespace pkv
