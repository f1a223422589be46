// row_values.cuh -- conversions that the 4-bit and the 8-bit rows share (kv_q4.cu, kv_q8.cu).
#pragma once

#include <stdint.h>

namespace fanout {

// Two fp32 -> e4m3 (low byte: lo), saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f16_f32(uint32_t h2) {
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h2));
    return f;
}
__device__ __forceinline__ float hi_f16_f32(uint32_t h2) { return lo_f16_f32(h2 >> 16); }
// x / den rounded to nearest, from r = 1 / den rounded to nearest: the quotient's
// remainder is exact in one fused step, and adding its share rounds correctly
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990). |x| <= 512 den here, and den (gs, 6 gs, or a group scale times gs) is
// in [2e-33, 4.5e32]. A remainder is a multiple of the product of q's and den's last places:
// of 2^-57 den for the quotients that decide a code (2^-11 and up). Where den is small that
// would be less than the smallest subnormal, 2^-149, so there it is formed 2^64 times as
// large. (Without that a pool scale of 2^-99 - 2^-123 held 2^-109 as 0: the quotient, a step
// above the tie at 2^-10, came out as the tie.) kSmall: den may be below 2^-60, which pool
// scales of 2^-50 and more do not give; kernels for those leave it out (8192 rows of 8 heads
// in and out with it and without: 8 bits 17.0 and 16.2 us, 4 bits 22.6 and 21.4).
template <bool kSmall>
__device__ __forceinline__ float quotient(float x, float den, float r) {
    const bool small = kSmall && den < 0x1p-60f;
    const float up = small ? 0x1p64f : 1.f, down = small ? 0x1p-64f : 1.f;
    const float q = x * r;
    return fmaf(fmaf(-q, den * up, x * up), r * down, q);
}
inline bool small_scales(float k_scale, float v_scale) {
    return k_scale < 0x1p-50f || v_scale < 0x1p-50f;
}

}  // namespace fanout
