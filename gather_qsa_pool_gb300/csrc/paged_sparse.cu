// paged_sparse.cu -- attention of each token over the blocks listed for it, in place on a paged cache.
#include "paged.cuh"

namespace qsa {

cudaError_t launch_paged_sparse(const SparseArgs &a, cudaStream_t st)
{
    DenseArgs d;
    d.kv = a.kv;
    d.sv = a.sv;
    d.kv_dtype = a.kv_dtype;
    d.q_dtype = a.q_dtype;
    d.q = a.q;
    d.ld_q = a.ld_q;
    d.out = a.out;
    d.lse = a.lse;
    d.H_q = a.H_q;
    d.d = a.d;
    d.scale = a.scale;
    d.causal = 1;
    d.pool_rows = 0;
    d.list = {a.blocks, a.counts, a.k_blk};
    return launch_dense_attn(d, st);
}

}  // namespace qsa
