// kv_q8.cu -- rows into the 8-bit KV cache and back.
//
// A cached row is 128 e4m3 codes: with the pool's scale gs
//   code = e4m3(x / gs), value = code * gs,
// the quotient in fp32, rounded to nearest, ties to even, saturating at 448. A pool is
// [num_pages][H_kv][page][128] bytes, so a page of a KV head is a tile of 128-byte rows,
// which the attention kernel's products read as they are.
//
// A lane owns 16 values (32 bytes of bf16, 16 of codes); 8 lanes make a K row, 8 its V
// row, so a half-warp handles a (row, KV head) pair without exchanges and its stores are
// whole 128-byte lines. It takes two pairs at once, so that twice the bytes are under way
// (one: 26.5 us for 8192 rows of 8 heads in and out; four: 26.1, fewer warps fit), and loads
// a new row beside its slot. Two: 23.1 us for 101 MB (4.4 TB/s, the rows just written read
// from L2); the chain of slot, row and store and two ramps are what is left, and one call
// behind another, where those overlap (launch_after.cuh), it takes 16.2 (6.2 TB/s). 8 rows:
// a launch each, 2.0 us back to back in a graph.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch_after.cuh"
#include "ptx_fp8.cuh"
#include "ptx_sm100.cuh"
#include "row_values.cuh"
#include "rows.h"

namespace fanout {
namespace {

constexpr int kErrInval = 1;  // FANOUT_EINVAL
constexpr int kWarps = 8;
constexpr int kRows = 2;  // (row, head) pairs of a half-warp

// 256-bit load (address 32-byte aligned). An ordinary one: the rows may have been written
// while this kernel started up (launch_after.cuh).
__device__ __forceinline__ void load_v8(const void* ptr, uint32_t (&r)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "l"(ptr)
                 : "memory");
}

// Pair k of this half-warp; false behind the last one.
__device__ __forceinline__ bool row_of(const Q8RowParams& p, int k, uint32_t& r, uint32_t& h) {
    const uint32_t item =
        (blockIdx.x * kRows + k) * (2 * kWarps) + (threadIdx.x >> 4);  // < 2^31 + 32 (host check)
    r = item / static_cast<uint32_t>(p.H_kv);
    h = item - r * static_cast<uint32_t>(p.H_kv);
    return r < static_cast<uint32_t>(p.n_rows);
}
// The byte of the pools where the pair's row starts; false when there is nothing to do.
__device__ __forceinline__ bool place_of(const Q8RowParams& p, int64_t slot, uint32_t h,
                                         int64_t& at) {
    if (slot < 0) return false;  // a padded row
    if (slot >= p.n_slots) {
        if ((threadIdx.x & 15) == 0) atomicCAS(p.err, 0, kErrInval);
        return false;
    }
    const int64_t page = slot >> p.page_shift;
    const int32_t in_page = static_cast<int32_t>(slot) & ((1 << p.page_shift) - 1);
    at = ((((page * p.H_kv + h) << p.page_shift) + in_page) * kHD);
    return true;
}

template <bool kSmall>
__global__ void __launch_bounds__(32 * kWarps) append_q8_kernel(const Q8RowParams p) {
    after_previous();
    const int part = threadIdx.x & 7;
    const bool is_v = threadIdx.x & 8;
    uint32_t raws[kRows][8], hs[kRows];
    int64_t slot[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        uint32_t r;
        slot[k] = -1;
        if (!row_of(p, k, r, hs[k])) continue;
        slot[k] = __ldcg(p.slots + r);
        const __nv_bfloat16* src = is_v ? p.v_rows + static_cast<int64_t>(r) * p.v_stride
                                        : p.k_rows + static_cast<int64_t>(r) * p.k_stride;
        src += hs[k] * kHD + part * 16;
        if (p.align32) {  // one load of a whole sector
            load_v8(src, raws[k]);
        } else {
            const uint4* from = reinterpret_cast<const uint4*>(src);
            const uint4 a = __ldcg(from), b = __ldcg(from + 1);
            raws[k][0] = a.x, raws[k][1] = a.y, raws[k][2] = a.z, raws[k][3] = a.w;
            raws[k][4] = b.x, raws[k][5] = b.y, raws[k][6] = b.z, raws[k][7] = b.w;
        }
    }
    const float gs = is_v ? p.v_scale : p.k_scale, rcp = is_v ? p.v_rcp : p.k_rcp;
    const float most = 512.f * gs;  // (codes saturate at 448, so 512 stands for what is larger)
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        int64_t at;
        if (!place_of(p, slot[k], hs[k], at)) continue;
        uint32_t* raw = raws[k];
        uint32_t top2 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top2 = ptx::max_nan_bf16x2(top2, raw[i] & 0x7fff7fffu);
        if ((top2 & 0x7fffu) > 0x7f80u || (top2 >> 16) > 0x7f80u) {
            // a NaN is recorded, and held as 0: it must not reach other rows
            atomicCAS(p.err, 0, kErrInval);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if ((raw[i] & 0x7fffu) > 0x7f80u) raw[i] &= 0xffff0000u;
                if ((raw[i] & 0x7fff0000u) > 0x7f800000u) raw[i] &= 0xffffu;
            }
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t v = raw[2 * i + (c >> 1)];
                const float x = __uint_as_float(c & 1 ? v & 0xffff0000u : v << 16);
                // (a zero's sign does not pass the correction)
                y[c] = copysignf(quotient<kSmall>(fminf(fmaxf(x, -most), most), gs, rcp), x);
            }
            w[i] = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
        }
        *reinterpret_cast<uint4*>((is_v ? p.v_pool : p.k_pool) + at + part * 16) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__global__ void __launch_bounds__(32 * kWarps) read_q8_kernel(const Q8RowParams p) {
    after_previous();
    const int part = threadIdx.x & 7;
    const bool is_v = threadIdx.x & 8;
    int64_t slot[kRows], at[kRows];
    uint32_t rs[kRows], hs[kRows];
    uint4 cs[kRows];
    bool on[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        slot[k] = -1;
        if (row_of(p, k, rs[k], hs[k])) slot[k] = __ldcg(p.slots + rs[k]);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        on[k] = place_of(p, slot[k], hs[k], at[k]);
        if (on[k])
            cs[k] = __ldcg(reinterpret_cast<const uint4*>((is_v ? p.v_pool : p.k_pool) + at[k] +
                                                         part * 16));
    }
    const float gs = is_v ? p.v_scale : p.k_scale;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        if (!on[k]) continue;
        const uint32_t w[4] = {cs[k].x, cs[k].y, cs[k].z, cs[k].w};
        uint32_t out[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a, b;
            ptx::f16x2_of_e4m3x4(w[i], a, b);
            out[2 * i] = ptx::pack_bf16x2(lo_f16_f32(a) * gs, hi_f16_f32(a) * gs);
            out[2 * i + 1] = ptx::pack_bf16x2(lo_f16_f32(b) * gs, hi_f16_f32(b) * gs);
        }
        __nv_bfloat16* dst = is_v ? p.v_out + static_cast<int64_t>(rs[k]) * p.v_stride
                                  : p.k_out + static_cast<int64_t>(rs[k]) * p.k_stride;
        dst += hs[k] * kHD + part * 16;
        if (p.align32) {
            ptx::st_global_v8(dst, out);
        } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
        }
    }
}

}  // namespace

cudaError_t launch_q8_rows(const Q8RowParams& p, bool read, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.n_rows) * p.H_kv;
    if (items <= 0) return cudaSuccess;
    const int grid = static_cast<int>((items + 2 * kWarps * kRows - 1) / (2 * kWarps * kRows));
    auto* kernel = read                                 ? read_q8_kernel
                   : small_scales(p.k_scale, p.v_scale) ? append_q8_kernel<true>
                                                        : append_q8_kernel<false>;
    return launch_after(kernel, grid, 32 * kWarps, 0, stream, p);
}

}  // namespace fanout
