// E4M3 codes of a KV pool: conversions shared by the slot pool's and the paged
// pool's kernels.
//
// Writing stores E4M3(x * inv_scale): the bfloat16 input widened,
// one float32 product, then the hardware's nearest-even conversion that
// saturates to the largest finite code (448).  Reading expands code c to
// bfloat16(value(c) * scale): E4M3 -> f16 is exact, the product is one
// float32 rounding, the bfloat16 rounding is to nearest even.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace unipin {

// two floats -> two E4M3 codes (lo in the low byte)
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// eight bfloat16 (16 bytes) -> eight E4M3 codes (8 bytes), x * inv each
__device__ __forceinline__ uint2 e4m3x8_from_bf16(uint4 x, float inv)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __fmul_rn(__uint_as_float(w[i] << 16), inv);
        const float hi = __fmul_rn(__uint_as_float(w[i] & 0xFFFF0000u), inv);
        c[i] = e4m3x2_from_f32(lo, hi);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// eight E4M3 codes -> eight bfloat16, value * scale each
__device__ __forceinline__ uint4 bf16x8_from_e4m3(uint2 codes, float scale)
{
    const uint32_t w[2] = {codes.x, codes.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t pair = (uint16_t)(w[i >> 1] >> ((i & 1) * 16));
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
        const float lo = __fmul_rn(__half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu))), scale);
        const float hi = __fmul_rn(__half2float(__ushort_as_half((unsigned short)(h2 >> 16))), scale);
        const uint32_t blo = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
        const uint32_t bhi = __bfloat16_as_ushort(__float2bfloat16_rn(hi));
        o[i] = blo | (bhi << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace unipin
