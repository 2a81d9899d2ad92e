// bqg_attn_launch.cuh -- host side of the attention kernel, one cache format per translation unit.
#pragma once

#include <algorithm>
#include <mutex>

#include "bqg_attn.cuh"

namespace bqg {

// Counters at the start of every workspace: the same bytes whatever the
// call's instantiation, so calls of different shapes can take turns on one.
constexpr int kAttnMaxCtas = 4096;
constexpr size_t kAttnCounterBytes = kAttnMaxCtas * sizeof(int);

// The workspace of a call: counters, partial rows, their maxima and sums.
struct AttnPlan {
    size_t ws_bytes;
};

inline cudaError_t take_error(int &word, int *out)
{
    int v = 0, zero = 0;
    if (cudaError_t e = cudaMemcpyFromSymbol(&v, word, sizeof(int))) return e;
    if (v)
        if (cudaError_t e = cudaMemcpyToSymbol(word, &zero, sizeof(int))) return e;
    *out = v;
    return cudaSuccess;
}

// rows: the most rows (new tokens x heads of a group) of any sequence.  Up
// to 16 one row tile, more two per CTA where the accumulators fit in
// registers (head_dim <= 128), so that a row of the cache is read from L2
// once for each 32 rows.
template <int FMT> AttnFn attn_pick(int D, int rows)
{
    if (D == 64) return rows <= 16 ? attn_fn<FMT, 64, 1>() : attn_fn<FMT, 64, 2>();
    if (D == 128) return rows <= 16 ? attn_fn<FMT, 128, 1>() : attn_fn<FMT, 128, 2>();
    return attn_fn<FMT, 256, 1>();
}

// Plans the call (plan) or, plan null, launches it.
template <int FMT>
cudaError_t attn_launch(const AttnParams &params, int D, int rows, int &error_word, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    const AttnFn fn = attn_pick<FMT>(D, rows);
    // occupancy of each instantiation, once per device
    static std::mutex mu;
    static int occ[64][6];
    int dev = 0, sms = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) return e;
    const int which = (D == 64 ? 0 : D == 128 ? 2 : 4) + (fn.rows > 16);
    int n = 0;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (occ[dev][which] == 0) {
            if (cudaError_t e = cudaFuncSetAttribute(fn.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, fn.smem)) return e;
            int k = 0;
            if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, fn.kern, 32 * kAttnWarps, fn.smem)) return e;
            if (k < 1) return cudaErrorLaunchOutOfResources;
            occ[dev][which] = k;
        }
        n = occ[dev][which];
    }
    const int ctas = std::min(sms * n, kAttnMaxCtas);                     // all resident at once
    if (plan) {
        plan->ws_bytes = kAttnCounterBytes + (size_t)2 * ctas * fn.rows * (D + 2) * sizeof(float);
        return cudaSuccess;
    }
    void *word = nullptr;
    if (cudaError_t e = cudaGetSymbolAddress(&word, error_word)) return e;
    AttnParams p = params;
    p.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.counters) + kAttnCounterBytes);
    // never more CTAs than units could exist
    const int64_t cap = std::min<int64_t>(p.max_pages << p.cache.lp, 0x7fff0000);
    const int64_t per_row_tile = (cap + kUnit - 1) / kUnit;
    const int64_t row_tiles = ((int64_t)p.max_q * p.group + fn.rows - 1) / fn.rows;
    const double most = (double)p.n_seq * p.cache.n_kv * (double)row_tiles * (double)per_row_tile;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(1.0, std::min((double)ctas, most)));
    cfg.blockDim = dim3(32 * kAttnWarps);
    cfg.dynamicSmemBytes = fn.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn.kern, p, (int *)word);
}

}  // namespace bqg
