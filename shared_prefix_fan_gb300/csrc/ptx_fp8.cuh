// ptx_fp8.cuh -- inline-PTX wrappers for 8-bit floats (e4m3): the tensor core's product of
// e4m3 tiles, and conversions between e4m3 and f16. Encodings follow the public PTX ISA
// (tcgen05 kind::f8f6f4 instruction descriptor).
#pragma once

#include <stdint.h>

namespace fanout {
namespace ptx {

// kind::f8f6f4 instruction descriptor: D fp32, A and B e4m3 (formats 0), both K-major,
// dense; fields as in idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T over 32 values of K, run by a whole warp and issued by
// the lane whose `leader` is 1.
__device__ __forceinline__ void mma_e4m3_ss_if(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                               uint32_t idesc, uint32_t accumulate,
                                               uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

// Four e4m3 bytes to two f16 pairs (exact).
__device__ __forceinline__ void f16x2_of_e4m3x4(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
}

// Four f16 values (two pairs) as e4m3, and what is left of them, as e4m3 too (the
// difference is exact: both are multiples of f16's step at the value).
__device__ __forceinline__ void split_e4m3x4(uint32_t a, uint32_t b, uint32_t& upper, uint32_t& rest) {
    asm("{\n\t.reg .b16 u0, u1, r0, r1;\n\t"
        ".reg .b32 h0, h1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 u0, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 u1, %3;\n\t"
        "cvt.rn.f16x2.e4m3x2 h0, u0;\n\t"
        "cvt.rn.f16x2.e4m3x2 h1, u1;\n\t"
        "sub.rn.f16x2 h0, %2, h0;\n\t"
        "sub.rn.f16x2 h1, %3, h1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 r0, h0;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 r1, h1;\n\t"
        "mov.b32 %0, {u0, u1};\n\t"
        "mov.b32 %1, {r0, r1};\n\t}"
        : "=r"(upper), "=r"(rest)
        : "r"(a), "r"(b));
}

}  // namespace ptx
}  // namespace fanout
