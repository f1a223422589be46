// attn_rows_q8.cu -- attn_rows.cuh over 8-bit pools, tokens in causal order.
#include "attn_rows.cuh"

namespace fanout {

cudaError_t launch_attn_rows_q8(const RowParams& p, const CUtensorMap& tm_q,
                                const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid,
                                cudaStream_t stream) {
    return p.nq == 2 ? launch_nq<2, Pool::q8, false>(p, tm_q, tm_k, tm_v, grid, stream)
                     : launch_nq<1, Pool::q8, false>(p, tm_q, tm_k, tm_v, grid, stream);
}

}  // namespace fanout
