// attn_tree.cu -- attn_rows.cuh for trees of drafted tokens, over all three kinds of pools.
#include "attn_rows.cuh"

namespace fanout {
namespace {

template <Pool F>
cudaError_t launch_tree(const RowParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                        const CUtensorMap& tm_v, int grid, cudaStream_t stream) {
    return p.nq == 2 ? launch_nq<2, F, true>(p, tm_q, tm_k, tm_v, grid, stream)
                     : launch_nq<1, F, true>(p, tm_q, tm_k, tm_v, grid, stream);
}

}  // namespace

cudaError_t launch_attn_tree(const RowParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, Pool pool, int grid, cudaStream_t stream) {
    return pool == Pool::q8   ? launch_tree<Pool::q8>(p, tm_q, tm_k, tm_v, grid, stream)
           : pool == Pool::q4 ? launch_tree<Pool::q4>(p, tm_q, tm_k, tm_v, grid, stream)
                              : launch_tree<Pool::bf16>(p, tm_q, tm_k, tm_v, grid, stream);
}

}  // namespace fanout
