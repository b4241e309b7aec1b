// 8-bit values (e4m3) of a cache with scales: conversions, which round to
// the nearest (ties to even) and take what is beyond the range to the largest.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "clk_mma.cuh"

namespace clk {

// Two values as codes, `a` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Two codes (the low 16 bits) as float16, which holds them exactly.
__device__ __forceinline__ uint32_t half_of_e4m3(uint32_t codes)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}

__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

__device__ __forceinline__ float from_e4m3(uint8_t code) { return halves(half_of_e4m3(code)).x; }

__device__ __forceinline__ void from_e4m3x4(uint32_t codes, float* f)
{
    const float2 a = halves(half_of_e4m3(codes)), b = halves(half_of_e4m3(codes >> 16));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

// The least power of two (at least 2^-120) with which `top` is at most 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float top)
{
    constexpr int least = 127 - 120;
    const uint32_t bits = __float_as_uint(top);
    int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < least) e = least;
    return __uint_as_float((uint32_t)e << 23);
}

// Eight codes as elements of the products' type, times their scale: rounded once (exact for scales that are powers
// of two in the type's range).  PLAIN: a scale that the type holds, which is `mult` twice.  (A product is then one
// instruction a pair, and the same: codes are exact in both types.)
template <bool BF16>
__device__ __forceinline__ bool fits(float scale)
{
    if (BF16) return (__float_as_uint(scale) & 0xffffu) == 0;
    return __half2float(__float2half_rn(scale)) == scale;
}

template <bool BF16, bool PLAIN>
__device__ __forceinline__ uint4 widen(uint2 codes, float scale, uint32_t mult)
{
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = half_of_e4m3((i < 2 ? codes.x : codes.y) >> 16 * (i & 1));
        const float2 f = halves(h);
        if (!PLAIN) {
            y[i] = pack2<BF16>(f.x * scale, f.y * scale);
        } else if (BF16) {
            const uint32_t w = pack2<true>(f.x, f.y);
            const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&mult));
            y[i] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
            const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&mult));
            y[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
}

}  // namespace clk
