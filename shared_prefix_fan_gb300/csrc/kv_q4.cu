// kv_q4.cu -- rows into the 4-bit KV cache and back.
//
// A cached row of 128 values is 8 groups of 16. With the pool's scale gs and a
// group's largest magnitude a:
//   sc   = e4m3(a / (6 gs))            (1 byte, saturating at 448)
//   code = e2m1(x / (sc gs))           (4 bits: 0, .5, 1, 1.5, 2, 3, 4, 6 and signs)
//   value = e2m1(code) * (sc gs)
// each rounded to nearest, ties to even, the quotients in fp32. A group whose
// scale rounds to 0 holds zeros. 64 bytes of codes and 8 of scales per row, so
// a (page, KV head) block is page * 64 code bytes, then page * 8 scale bytes.
// Eight values share a 32-bit word: values 0, 2, 4, 6 in the low half (4 bits
// each, from bit 0 up), 1, 3, 5, 7 in the high half, so that one shift brings a
// pair of neighbours to the same place of both halves of a register, which is
// how the attention kernel widens them.
//
// One warp per (row, KV head): lanes 0..15 its K row, lanes 16..31 its V row,
// 8 values (16 bytes of bf16, one code word) a lane; two lanes share a group.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fanout_internal.h"

namespace fanout {
namespace {

constexpr int kErrInval = 1;  // FANOUT_EINVAL

// Two fp32 -> e4m3 (low byte: lo), saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(byte)));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h2));
    return f;
}
// Eight fp32 -> a code word (the order above).
__device__ __forceinline__ uint32_t e2m1_word(const float (&y)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %3, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %7, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %4, %2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %6;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return w;
}
// e2m1 code (4 bits) -> fp32.
__device__ __forceinline__ float e2m1_f32(uint32_t code) {
    const uint32_t m = code & 7u;
    // magnitudes below 2 are code / 2; from 2 on, exponent and half step as stored
    const float a = m < 4 ? 0.5f * static_cast<float>(m)
                          : static_cast<float>((2u + (m & 1u)) << ((m >> 1) - 2u));
    return (code & 8u) ? -a : a;
}

struct Place {
    int64_t codes, scales;  // byte offsets of the row in the pool
};
__device__ __forceinline__ Place place_of(const Q4RowParams& p, int64_t slot, int32_t h) {
    const int64_t page = slot >> p.page_shift;
    const int32_t off = static_cast<int32_t>(slot) & ((1 << p.page_shift) - 1);
    const int64_t block = (page * p.H_kv + h) * (static_cast<int64_t>(kQ4RowBytes) << p.page_shift);
    return {block + off * 64, block + (static_cast<int64_t>(64) << p.page_shift) + off * 8};
}

__global__ void __launch_bounds__(256) append_q4_kernel(const Q4RowParams p) {
    const int lane = threadIdx.x & 31, part = lane & 15;
    const bool is_v = lane >= 16;
    const int64_t items = static_cast<int64_t>(p.n_rows) * p.H_kv;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    const float gs = is_v ? p.v_scale : p.k_scale;
    const float c6 = 6.0f * gs;
    for (int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
         item < items; item += warps) {
        const int64_t r = item / p.H_kv;
        const int32_t h = static_cast<int32_t>(item - r * p.H_kv);
        const int64_t slot = p.slots[r];
        if (slot < 0) continue;  // a padded row
        if (slot >= p.n_slots) {
            if (lane == 0) atomicCAS(p.err, 0, kErrInval);
            continue;
        }
        const __nv_bfloat16* src = is_v ? p.v_rows + r * p.v_stride : p.k_rows + r * p.k_stride;
        const uint4 raw = *reinterpret_cast<const uint4*>(src + h * kHD + part * 8);
        float x[8] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                      __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u),
                      __uint_as_float(raw.z << 16), __uint_as_float(raw.z & 0xffff0000u),
                      __uint_as_float(raw.w << 16), __uint_as_float(raw.w & 0xffff0000u)};
        float top = 0.f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (isnan(x[i])) {  // recorded, and held as 0: it must not reach other rows
                nan = true;
                x[i] = 0.f;
            }
            top = fmaxf(top, fabsf(x[i]));
        }
        if (nan) atomicCAS(p.err, 0, kErrInval);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const uint32_t sc = e4m3x2(__fdiv_rn(top, c6), 0.f) & 0xffu;
        const float den = e4m3_f32(sc) * gs;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = den > 0.f ? __fdiv_rn(x[i], den) : 0.f;
        const Place at = place_of(p, slot, h);
        uint8_t* pool = is_v ? p.v_pool : p.k_pool;
        *reinterpret_cast<uint32_t*>(pool + at.codes + part * 4) = e2m1_word(y);
        if ((part & 1) == 0) pool[at.scales + (part >> 1)] = static_cast<uint8_t>(sc);
    }
}

__global__ void __launch_bounds__(256) read_q4_kernel(const Q4RowParams p) {
    const int lane = threadIdx.x & 31, part = lane & 15;
    const bool is_v = lane >= 16;
    const int64_t items = static_cast<int64_t>(p.n_rows) * p.H_kv;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    const float gs = is_v ? p.v_scale : p.k_scale;
    for (int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
         item < items; item += warps) {
        const int64_t r = item / p.H_kv;
        const int32_t h = static_cast<int32_t>(item - r * p.H_kv);
        const int64_t slot = p.slots[r];
        if (slot < 0) continue;
        if (slot >= p.n_slots) {
            if (lane == 0) atomicCAS(p.err, 0, kErrInval);
            continue;
        }
        const Place at = place_of(p, slot, h);
        const uint8_t* pool = is_v ? p.v_pool : p.k_pool;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(pool + at.codes + part * 4);
        const float den = e4m3_f32(pool[at.scales + (part >> 1)]) * gs;
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = e2m1_f32((w >> (4 * i)) & 15u) * den;
            const float b = e2m1_f32((w >> (16 + 4 * i)) & 15u) * den;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[i]) : "f"(b), "f"(a));
        }
        __nv_bfloat16* dst = is_v ? p.v_out + r * p.v_stride : p.k_out + r * p.k_stride;
        *reinterpret_cast<uint4*>(dst + h * kHD + part * 8) =
            make_uint4(out[0], out[1], out[2], out[3]);
    }
}

}  // namespace

cudaError_t launch_q4_rows(const Q4RowParams& p, bool read, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.n_rows) * p.H_kv;
    if (items <= 0) return cudaSuccess;
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t blocks = (items + 7) / 8;
    const int grid = static_cast<int>(blocks < 8LL * sms ? blocks : 8LL * sms);
    if (read) read_q4_kernel<<<grid, 256, 0, stream>>>(p);
    else append_q4_kernel<<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fanout
