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
// A lane owns one group: 16 values (32 bytes of bf16), two code words and a scale;
// 8 lanes make a K row, 8 its V row, so a warp handles two (row, KV head) pairs in
// one pass, without exchanges. The floor of many rows is HBM's (656 bytes a pair of K and
// V rows): 32 bytes a lane keep enough reads in flight (with 16, and a row
// per warp, 8192 rows of 8 heads took 33 us in and out), and the work per value is
// kept short: the quotients are products with the reciprocal, corrected (quotient,
// below), the largest magnitude comes from packed maxima, codes from the e2m1
// conversions (with fp32 divisions it took 47 us). Measured: 8192 rows of 8 heads in
// and out 26.6 us (86 MB: 3.2 TB/s, the rows just written read from L2; what its warps
// wait for is loads, one dependent chain a lane), 8 rows 10 us (two launches).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fanout_internal.h"
#include "ptx_sm100.cuh"
#include "row_values.cuh"

namespace fanout {
namespace {

constexpr int kErrInval = 1;  // FANOUT_EINVAL
constexpr int kWarps = 8;

__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
    return lo_f16_f32(ptx::f16x2_of_e4m3x2(byte));
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
struct Place {
    int64_t codes, scales;  // byte offsets of the row in the pool
};
__device__ __forceinline__ Place place_of(const Q4RowParams& p, int64_t slot, int32_t h) {
    const int64_t page = slot >> p.page_shift;
    const int32_t off = static_cast<int32_t>(slot) & ((1 << p.page_shift) - 1);
    const int64_t block = (page * p.H_kv + h) * (static_cast<int64_t>(kQ4RowBytes) << p.page_shift);
    return {block + off * 64, block + (static_cast<int64_t>(64) << p.page_shift) + off * 8};
}

// The (row, head) pair of this half-warp and its slot; false when there is nothing
// to do.
__device__ __forceinline__ bool item_of(const Q4RowParams& p, uint32_t& r, uint32_t& h,
                                        int64_t& slot) {
    const uint32_t item = blockIdx.x * (2 * kWarps) + (threadIdx.x >> 4);  // < 2^31 + 16 (host check)
    r = item / static_cast<uint32_t>(p.H_kv);
    h = item - r * static_cast<uint32_t>(p.H_kv);
    if (r >= static_cast<uint32_t>(p.n_rows)) return false;
    slot = __ldg(p.slots + r);
    if (slot < 0) return false;  // a padded row
    if (slot >= p.n_slots) {
        if ((threadIdx.x & 15) == 0) atomicCAS(p.err, 0, kErrInval);
        return false;
    }
    return true;
}

template <bool kSmall>
__global__ void __launch_bounds__(32 * kWarps) append_q4_kernel(const Q4RowParams p) {
    const int group = threadIdx.x & 7;
    const bool is_v = threadIdx.x & 8;
    uint32_t r, h;
    int64_t slot;
    if (!item_of(p, r, h, slot)) return;
    const __nv_bfloat16* src = is_v ? p.v_rows + static_cast<int64_t>(r) * p.v_stride
                                    : p.k_rows + static_cast<int64_t>(r) * p.k_stride;
    uint32_t raw[8];
    src += h * kHD + group * 16;
    if (p.align32) {  // one load of a whole sector
        ptx::ld_global_v8(src, raw);
    } else {
        const uint4* from = reinterpret_cast<const uint4*>(src);
        const uint4 a = __ldg(from), b = __ldg(from + 1);
        raw[0] = a.x, raw[1] = a.y, raw[2] = a.z, raw[3] = a.w;
        raw[4] = b.x, raw[5] = b.y, raw[6] = b.z, raw[7] = b.w;
    }
    // largest magnitude; a NaN among the values shows in it
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top2 = ptx::max_nan_bf16x2(top2, raw[i] & 0x7fff7fffu);
    if ((top2 & 0x7fffu) > 0x7f80u || (top2 >> 16) > 0x7f80u) {
        // recorded, and held as 0: it must not reach other rows
        atomicCAS(p.err, 0, kErrInval);
        top2 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if ((raw[i] & 0x7fffu) > 0x7f80u) raw[i] &= 0xffff0000u;
            if ((raw[i] & 0x7fff0000u) > 0x7f800000u) raw[i] &= 0xffffu;
            top2 = ptx::max_nan_bf16x2(top2, raw[i] & 0x7fff7fffu);
        }
    }
    const float top = fmaxf(__uint_as_float(top2 << 16), __uint_as_float(top2 & 0xffff0000u));
    const float gs = is_v ? p.v_scale : p.k_scale;
    // (from 448 on the scale saturates, so 512 stands for whatever is larger)
    const float c6 = 6.0f * gs;
    const float most = quotient<kSmall>(fminf(top, 512.f * c6), c6, is_v ? p.v_rcp6 : p.k_rcp6);
    const uint32_t sc = e4m3x2(most, 0.f) & 0xffu;
    const float den = e4m3_f32(sc) * gs;
    uint32_t w[2] = {0u, 0u};
    if (sc > 0) {
        const float rcp = __frcp_rn(den);
        if (sc >= 0x7e) {
            // saturated: whatever is above 8 den (infinity too) has code 6, as 8 den has
            const float most = 8.f * den;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float lo = fminf(fmaxf(__uint_as_float(raw[i] << 16), -most), most);
                const float hi = fminf(fmaxf(__uint_as_float(raw[i] & 0xffff0000u), -most), most);
                raw[i] = (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v = raw[4 * half + (i >> 1)];
                const float x = __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16);
                y[i] = quotient<kSmall>(x, den, rcp);
            }
            w[half] = e2m1_word(y);
        }
    }
    const Place at = place_of(p, slot, h);
    uint8_t* pool = is_v ? p.v_pool : p.k_pool;
    *reinterpret_cast<uint2*>(pool + at.codes + group * 8) = make_uint2(w[0], w[1]);
    pool[at.scales + group] = static_cast<uint8_t>(sc);
}

__global__ void __launch_bounds__(32 * kWarps) read_q4_kernel(const Q4RowParams p) {
    const int group = threadIdx.x & 7;
    const bool is_v = threadIdx.x & 8;
    uint32_t r, h;
    int64_t slot;
    if (!item_of(p, r, h, slot)) return;
    const Place at = place_of(p, slot, h);
    const uint8_t* pool = is_v ? p.v_pool : p.k_pool;
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(pool + at.codes + group * 8));
    const float den = e4m3_f32(__ldg(pool + at.scales + group)) * (is_v ? p.v_scale : p.k_scale);
    __nv_bfloat16* dst = is_v ? p.v_out + static_cast<int64_t>(r) * p.v_stride
                              : p.k_out + static_cast<int64_t>(r) * p.k_stride;
    dst += h * kHD + group * 16;
    uint32_t out[8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t v[4];  // values 0 2, 4 6, 1 3, 5 7
        ptx::f16x2_of_e2m1x8(half ? w.y : w.x, v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            out[4 * half + 2 * i] =
                ptx::pack_bf16x2(lo_f16_f32(v[i]) * den, lo_f16_f32(v[2 + i]) * den);
            out[4 * half + 2 * i + 1] =
                ptx::pack_bf16x2(hi_f16_f32(v[i]) * den, hi_f16_f32(v[2 + i]) * den);
        }
    }
    if (p.align32) {
        ptx::st_global_v8(dst, out);
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
}

}  // namespace

cudaError_t launch_q4_rows(const Q4RowParams& p, bool read, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.n_rows) * p.H_kv;
    if (items <= 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>((items + 2 * kWarps - 1) / (2 * kWarps));
    if (read) read_q4_kernel<<<grid, 32 * kWarps, 0, stream>>>(p);
    else if (small_scales(p.k_scale, p.v_scale)) append_q4_kernel<true><<<grid, 32 * kWarps, 0, stream>>>(p);
    else append_q4_kernel<false><<<grid, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fanout
