// Verification of drafted tokens (sm_103a): see draft_verify.cu.
#pragma once

#include "kda_common.cuh"

namespace kda {

struct VerifyArgs {
    const void *p, *p_last, *q, *q_last;
    int64_t p_ss, p_rs, pl_s, q_ss, q_rs, ql_s;   // strides in elements
    const int32_t *tokens, *parents;              // [n][R]
    const float *u, *u_next;                      // [n][R], [n]
    int32_t *path, *path_len, *next;              // [n][max_len], [n], [n]
    int32_t n, R, V, max_len;
    uint64_t wait_ns;                             // the limit of a wait between a session's CTAs
};
cudaError_t launch_verify(const VerifyArgs& a, int io_bf16, cudaStream_t s);

}  // namespace kda
