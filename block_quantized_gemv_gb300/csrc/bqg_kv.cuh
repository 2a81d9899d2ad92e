// bqg_kv.cuh -- the paged cache as the kernels see it, and its host-side parameters.
#pragma once

#include "bqg_common.cuh"

namespace bqg {

// One cache (include/bqgemv.h), with the page size as a shift.
struct KvCacheDev {
    uint8_t *k, *v;              // [n_pages][n_kv][page][row bytes]
    uint16_t *k_scale, *v_scale; // [n_pages][n_kv][page][head_dim / 32] fp16 bits
    int64_t n_pages;
    int n_kv, lp;                // page = 1 << lp
};

// Bytes of one head's cached row.
template <int FMT, int D> struct KvRow {
    static constexpr int BYTES = (FMT == BQG_BF16) ? 2 * D : (FMT == BQG_Q8_0) ? D : D / 2;
    static constexpr int NB = D / QK;                     // blocks (quantized formats)
};

// Row number of (slot, head): rows of `row bytes` (and of D / 32 scales).
__device__ __forceinline__ int64_t kv_row(const KvCacheDev &c, int64_t slot, int head)
{
    const int64_t page = slot >> c.lp, at = slot & ((1 << c.lp) - 1);
    return ((page * c.n_kv + head) << c.lp) + at;
}
// `slot` is a place of the cache (not negative, not beyond its pages).
__device__ __forceinline__ bool kv_slot_ok(const KvCacheDev &c, int64_t slot) { return slot >= 0 && (slot >> c.lp) < c.n_pages; }

struct NormRopeParams {
    const void *q, *k, *v;
    int x_f32;
    int64_t q_stride, k_stride, v_stride;        // values between tokens
    int64_t T;
    int n_q, n_kv;                               // heads of q, of k and v
    int norm;
    const float *gamma_q, *gamma_k;
    float eps;
    const int32_t *pos;
    const float *table;
    int64_t n_pos;
    int rot, interleaved;                        // rot = 0: no rotation
    uint16_t *q_out, *k_out;                     // bf16; k_out null: keys go into the cache
    const int64_t *slots;                        // null: no cache
    KvCacheDev cache;
    int *error;                                  // device_error_word, set by the launch
};

struct KvReadParams {
    KvCacheDev cache;
    const int64_t *slots;
    int64_t T;
    void *k_out, *v_out;
    int *error;                                  // as above
};

cudaError_t launch_norm_rope(NormRopeParams p, int fmt, int D, int sms, cudaStream_t s, bool pdl);
cudaError_t launch_kv_read(KvReadParams p, int fmt, int D, int out_f32, int sms, cudaStream_t s, bool pdl);
// The error word of the current device for the cache's and attention's kernels (bits BQG_DEVERR_*, and those of bounded
// waits): the prefill GEMM's, so that bqg_last_device_error has no more words to fetch (each costs it 9 us).
cudaError_t device_error_word(int **out);

}  // namespace bqg
