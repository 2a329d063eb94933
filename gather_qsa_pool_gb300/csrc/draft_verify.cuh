// draft_verify.cuh -- launcher of the draft verification (draft_verify.cu); arguments are
// already validated.
#pragma once

#include "qsa_internal.cuh"

namespace qsa {

cudaError_t launch_draft_verify(const float *target, int64_t ld_t, const float *draft, int64_t ld_d,
                                const int32_t *tokens, const int32_t *n_draft, const float *u,
                                int64_t n_seq, int64_t max_draft, int64_t vocab, int32_t *tokens_out,
                                int32_t *n_accepted, cudaStream_t st);

}  // namespace qsa
