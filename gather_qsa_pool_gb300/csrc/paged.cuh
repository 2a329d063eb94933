// paged.cuh -- launchers of the paged cache's write and read (paged_rw.cu), for the C entry
// points; arguments are already validated.
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

}  // namespace qsa
