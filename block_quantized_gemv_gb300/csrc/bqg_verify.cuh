// bqg_verify.cuh -- verification of drafted tokens: parameters (include/bqgemv.h, bqg_tree_verify).
#pragma once

#include "bqg_kv.cuh"

namespace bqg {

struct VerifyParams {
    const void *target, *draft;          // [n_tokens][vocab], bf16 or fp32; draft null: chosen drafts
    int64_t target_stride, draft_stride;
    int vocab;
    const int32_t *tokens, *parent;      // parent null: a chain
    const int32_t *q_start;
    int n_seq;
    int64_t n_tokens;
    int max_q;
    const float *u;
    int32_t *n_accepted, *path, *next_token;
    int *error;                          // device_error_word, set by the launch
};

cudaError_t launch_verify(VerifyParams p, int x_f32, int sms, cudaStream_t s, bool pdl);

}  // namespace bqg
