// tg_block_scale.cuh - the power-of-two scale of a block of 128 values and the packing of its 8-bit values: what the
// quantiser (tg_quant.cu) and the norm that writes an 8-bit copy (tg_norm.cu) share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

// The scale of a block whose largest magnitude has fp32 bits `a`, and its reciprocal.  A
// block with a value that is not finite gets s = NaN and q = 0: the product of such a
// block is NaN, so the fault stays visible.
__device__ __forceinline__ void block_scale(uint32_t a, int top_exp, float& s, float& inv) {
    if (a >= 0x7f800000u) {
        s = __uint_as_float(0x7fc00000u);
        inv = 0.0f;
        return;
    }
    int j = static_cast<int>(a >> 23) - 127 - top_exp + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (j < -126) j = -126;
    if (a == 0u) j = 0;
    s = __uint_as_float(static_cast<uint32_t>(127 + j) << 23);
    inv = __uint_as_float(static_cast<uint32_t>(127 - j) << 23);
}

// Four values, scaled and rounded to 8 bits
template <bool E5M2>
__device__ __forceinline__ uint32_t pack8(float a, float b, float c, float d) {
    uint16_t lo, hi;
    if constexpr (E5M2) {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    return lo | static_cast<uint32_t>(hi) << 16;
}

}  // namespace tg
