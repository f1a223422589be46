// attn_q4.cu -- fan-out attention over a cache held in 4 bits.
//
// The rows of a cache (kv_q4.cu) are e2m1 codes with one e4m3 scale per 16
// values; out = softmax(scale q K^T) V over the values they stand for.
//
// One warp per query row (token, head): every lane holds 4 of the 128
// dimensions, keys are swept one by one with the online softmax (running
// maximum m and sum l in base 2, O rescaled when m moves), split over the
// planner's units and merged from their partials (m, l, O).
#include <cuda_bf16.h>

#include "fanout_internal.h"
#include "ptx_sm100.cuh"
#include "row_unit.cuh"

namespace fanout {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float e2m1_f32(uint32_t code) {
    const uint32_t m = code & 7u;
    const float a = m < 4 ? 0.5f * static_cast<float>(m)
                          : static_cast<float>((2u + (m & 1u)) << ((m >> 1) - 2u));
    return (code & 8u) ? -a : a;
}
__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(byte)));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}"
        : "=f"(f)
        : "r"(h2));
    return f;
}

// This lane's 4 values (dimensions 4 lane ..) of token slot `slot` of a block.
__device__ __forceinline__ void load4(const uint8_t* block, int page_size, int slot, int lane,
                                      float (&x)[4]) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(block + slot * 64) + (lane >> 1));
    const float s = e4m3_f32(__ldg(block + page_size * 64 + slot * 8 + (lane >> 2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * (lane & 1) + i;
        x[i] = e2m1_f32((w >> (16 * (e & 1) + 4 * (e >> 1))) & 15u) * s;
    }
}

__global__ void __launch_bounds__(32 * kWarps) attn_q4_kernel(const SplitParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ps = p.page_size;
    for (int ui = p.cta_first[blockIdx.x]; ui < p.cta_first[blockIdx.x + 1]; ++ui) {
        const Unit u = p.units[ui];
        const int32_t* table = p.page_table + static_cast<int64_t>(u.branch) * p.max_pages;
        for (int row = warp; row < u.n_tok * p.G; row += kWarps) {
            const int tok = u.tok_begin + row / p.G, hq = u.kv_head * p.G + row % p.G;
            const int64_t orow = static_cast<int64_t>(tok) * p.H_q + hq;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + orow * kHD + 4 * lane;
            float qf[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[i] = __bfloat162float(q[i]) * p.scale_log2;
            const int pos = p.tok_pos[tok];
            const int lo = pos - p.window + 1;
            for (int run = u.pos_base > 0 ? 0 : 1; run < 2; ++run) {
                const int begin = run == 0 ? first_begin(u, p.split_at) : u.key_begin;
                const int end = min(run == 0 ? u.pos_base : u.key_end, pos + 1);
                const int sinks = run == 0 || u.pos_base == 0 ? p.sinks : 0;
                for (int j = begin; j < end; ++j) {
                    if (j < lo && j >= sinks) continue;
                    const int64_t page = checked_page(p, table[j / ps]);
                    const int64_t block = (page * p.H_kv + u.kv_head) * (ps * kQ4RowBytes);
                    float k[4], v[4];
                    load4(p.k_pool + block, ps, j % ps, lane, k);
                    load4(p.v_pool + block, ps, j % ps, lane, v);
                    float s = k[0] * qf[0] + k[1] * qf[1] + k[2] * qf[2] + k[3] * qf[3];
                    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                    const float m_new = fmaxf(m, s);
                    const float corr = ptx::ex2(m - m_new), e = ptx::ex2(s - m_new);
                    l = l * corr + e;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = o[i] * corr + e * v[i];
                    m = m_new;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= p.o_scale;
            if (u.part >= 0) {
                const int i = row / p.G;
                const int64_t prow = static_cast<int64_t>(u.part) * (kBM * p.nq) +
                                     i / p.tpt * kBM + i % p.tpt * p.G + row % p.G;
                reinterpret_cast<float4*>(p.part_o + prow * kHD)[lane] =
                    make_float4(o[0], o[1], o[2], o[3]);
                if (lane == 0) p.part_ml[prow] = make_float2(m, l);
                continue;
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            if (p.out_bf16)
                reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * kHD)[lane] =
                    make_uint2(ptx::pack_bf16x2(o[0] * inv, o[1] * inv),
                               ptx::pack_bf16x2(o[2] * inv, o[3] * inv));
            else
                reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow * kHD)[lane] =
                    make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
            if (p.lse && lane == 0) p.lse[orow] = (m + __log2f(l)) * 0.69314718055994531f;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace

cudaError_t launch_attn_q4(const SplitParams& p, const CUtensorMap& /*tm_q*/, int grid,
                           cudaStream_t stream) {
    attn_q4_kernel<<<grid, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fanout
