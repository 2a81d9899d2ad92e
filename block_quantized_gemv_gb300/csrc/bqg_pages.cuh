// bqg_pages.cuh -- cached tokens moved and sequences branched: parameters (include/bqgemv.h).
#pragma once

#include "bqg_kv.cuh"

namespace bqg {

struct CompactParams {
    KvCacheDev cache;
    const int32_t *table;                // [n_seq][max_pages]
    int64_t max_pages;
    const int32_t *ctx_len, *path, *n_path;
    int n_seq, max_q;
    int32_t *ctx_out;                    // null: not wanted
    bool ctx_in_table;                   // some of it lies in the table, which other CTAs read: written by a launch of its own
    int slices;                          // CTAs per sequence
    int *error;                          // device_error_word, set by the launch
};

struct ForkParams {
    KvCacheDev cache;
    int32_t *table;                      // [n_rows][max_pages]
    int64_t max_pages;
    int n_rows;
    int32_t *ctx_len;
    const int32_t *parent, *child, *fresh;
    int n;
    int slices;                          // CTAs per branch
    int *error;
};

cudaError_t launch_compact(CompactParams p, int fmt, int D, int sms, cudaStream_t s, bool pdl);
cudaError_t launch_fork(ForkParams p, int fmt, int D, int sms, cudaStream_t s, bool pdl);

}  // namespace bqg
