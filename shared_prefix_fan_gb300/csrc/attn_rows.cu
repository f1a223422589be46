// attn_rows.cu -- attn_rows.cuh over bf16 and 4-bit pools, tokens in causal order.
#include "attn_rows.cuh"

namespace fanout {

cudaError_t launch_attn_rows(const RowParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, int grid, cudaStream_t stream) {
    return p.nq == 2 ? launch_nq<2, Pool::bf16, false>(p, tm_q, tm_k, tm_v, grid, stream)
                     : launch_nq<1, Pool::bf16, false>(p, tm_q, tm_k, tm_v, grid, stream);
}

cudaError_t launch_attn_rows_q4(const RowParams& p, const CUtensorMap& tm_q, int grid,
                                cudaStream_t stream) {
    const CUtensorMap none{};
    return p.nq == 2 ? launch_nq<2, Pool::q4, false>(p, tm_q, none, none, grid, stream)
                     : launch_nq<1, Pool::q4, false>(p, tm_q, none, none, grid, stream);
}

}  // namespace fanout
