// paged8.cuh -- rows of 8-bit pages: e4m3 codes and one power-of-two scale per
// row, kept as a biased exponent: a value is code * 2^(byte - 127).  The byte is the
// smallest with which the row's largest magnitude is at most 448, e4m3's largest
// number.  Such a scale is exact to apply (the codes' steps are relative, so a finer
// one would only move where they turn subnormal, 2^-15 below the largest), and
// every value that a row stands for is a bf16 number.
#pragma once

#include <cuda_fp8.h>

#include "vc_common.cuh"

namespace vc {
namespace paged {

// The least byte leaves the smallest code a normal number (2^-9 * 2^(10 - 127) =
// 2^-126), the largest keeps 448 * 2^(246 - 127) finite.
constexpr int kLeastScale = 10, kMostScale = 246;

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// amax = m 2^x, 1 <= m < 2: 448 = 1.75 * 2^8, so x - 8 where m <= 1.75, else x - 7:
// the addition carries into the exponent where the mantissa is above 0x600000.
// Rows past 448 * 2^119 (3e38) saturate.
__device__ __forceinline__ uint32_t scale_byte(float amax)
{
    const int b = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;
    return (uint32_t)min(max(b, kLeastScale), kMostScale);
}

// what values are multiplied with to become codes: 2^(127 - byte)
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return scale_of(254u - byte); }

// 8 values, already scaled, to codes (round to nearest, ties to even)
__device__ __forceinline__ uint2 encode8(const float2 (&x)[4])
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __nv_cvt_float2_to_fp8x2(x[i], __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// two codes (the low 16 bits), not yet scaled
__device__ __forceinline__ float2 decode2(uint32_t codes)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace paged
}  // namespace vc
