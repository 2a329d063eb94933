// paged.cuh -- launchers of the paged cache's write and read (paged_rw.cu), of appends with the
// rotation on the way (paged_append.cu) and of the sparse attention over it (paged_sparse.cu), for
// the C entry points; arguments are already validated.
#pragma once

#include "dense.cuh"

namespace qsa {

cudaError_t launch_paged_write(const void *k, const void *v, qsa_dtype src_dtype, int64_t ld_k,
                               int64_t ld_v, int d, const SeqView &sv, const KvView &kv,
                               qsa_dtype cache_dtype, cudaStream_t st);

cudaError_t launch_paged_read(const KvView &kv, qsa_dtype cache_dtype, int d, const int32_t *seq,
                              const int32_t *kv_len, int64_t n_seq, const int32_t *pos,
                              const int32_t *n_cells, int64_t n_list, int64_t max_cells, void *K_out,
                              void *V_out, qsa_dtype out_dtype, cudaStream_t st);

// The same as the write, and queries (NULL: none) and keys rotated on the way: the first `rot` values of each
// head (0: none), a multiple of 16, with frequencies base^(-2 i / rot).  Writes a 4-bit cache too.
cudaError_t launch_paged_append(const void *q, const void *k, const void *v, qsa_dtype src_dtype, int64_t ld_q,
                                int64_t ld_k, int64_t ld_v, int H_q, int d, int rot, double base, const int32_t *pos,
                                void *q_out, void *k_out, const SeqView &sv, const KvView &kv, qsa_dtype cache_dtype,
                                cudaStream_t st);

// Each token's attention over the blocks listed for it and its open block.
struct SparseArgs {
    KvView kv;
    SeqView sv;
    qsa_dtype kv_dtype, q_dtype;  // out has q's type
    const int32_t *blocks, *counts;
    int64_t k_blk;  // entries of a token's list
    const void *q;
    int64_t ld_q;
    void *out;
    float *lse;
    int H_q, d;
    float scale;
};
cudaError_t launch_paged_sparse(const SparseArgs &a, cudaStream_t st);

}  // namespace qsa
