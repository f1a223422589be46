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
// processor", 1990). |x| <= 512 den here, and den (6 gs, or a group scale times gs) is
// in [2e-33, 4.5e32]. Below about 2^-100 the remainder's last bits lie under the
// smallest subnormal: it is off by at most 2^-150, the quotient by 2^-41, where the
// quotients that decide a code (0.25 and up) have half steps of 2^-27 and more; with gs
// from 1e-30 to 1e-26, 6e6 random quotients all equal the division's.
__device__ __forceinline__ float quotient(float x, float den, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, den, x), r, q);
}

}  // namespace fanout
