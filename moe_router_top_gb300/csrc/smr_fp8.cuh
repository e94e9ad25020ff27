// smr_fp8.cuh -- a block's scale and codes in E4M3, for the quantisation kernels
// and for the gated product that writes its activations in E4M3.
//
// scale = amax / 448, codes = E4M3(x * (448 / amax)) rounded to nearest even,
// the quotients and the product in fp32. amax counts as 2^-110 at the least
// (448 / amax overflows below 2^-119 and every value would saturate); a block
// of zeros has scale 0 and codes +0. A block with a NaN or an infinity gets a
// NaN scale and codes +0.
#pragma once

#include "smr_device.cuh"

namespace smr {

// A block's scale and the factor for its values; m: the largest magnitude's
// bf16 bits (as unsigned integers magnitudes order like their values, with
// infinities and NaN above all). The factor is 0 for blocks of codes +0.
__device__ __forceinline__ void block_scale_e4m3(uint32_t m, float &scale, float &factor) {
    const float amax = fmaxf(__uint_as_float(m << 16), 0x1p-110f);
    scale = m == 0u ? 0.0f : (m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 448.0f));
    factor = m == 0u || m >= 0x7F80u ? 0.0f : __fdiv_rn(448.0f, amax);
}
__device__ __forceinline__ uint32_t abs_max8(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) m = max(m, max(w[u] & 0x7FFFu, (w[u] >> 16) & 0x7FFFu));
    return m;
}
// Eight values to codes (NaN times a factor of 0 is still NaN: those are cleared).
__device__ __forceinline__ uint2 codes8(const uint4 &v, float factor) {
    float f[8];
    unpack8(v, f);
    uint16_t h[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[u]) : "f"(f[2 * u + 1] * factor), "f"(f[2 * u] * factor));
    if (factor == 0.0f) return make_uint2(0u, 0u);
    return make_uint2((uint32_t)h[0] | (uint32_t)h[1] << 16, (uint32_t)h[2] | (uint32_t)h[3] << 16);
}

}  // namespace smr
