// bqg_attn_launch.cuh -- host side of the attention kernels, one cache format per translation unit.
#pragma once

#include <algorithm>
#include <mutex>

#include <cudaTypedefs.h>

#include "bqg_attn_tc.cuh"
#include "bqg_own.cuh"

namespace bqg {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// A workspace: the same bytes at its start whatever the call's kernel, so
// that calls of different shapes can take turns on one.  One arrival counter per
// CTA of the mma.sync kernel (zero between calls), then the sets
// that CTAs of the tcgen05 kernel share, then partial results.
constexpr int kAttnMaxCtas = 4096;
constexpr size_t kAttnCounterBytes = kAttnMaxCtas * sizeof(int);
constexpr size_t kAttnSetBytes = 1024 * sizeof(TcSet);
constexpr size_t kAttnHead = kAttnCounterBytes + kAttnSetBytes;

struct AttnPlan {
    size_t ws_bytes;
};

// Rows from which the tcgen05 kernel serves a call; below, the mma.sync kernel, which is built for one and two tiles of 8
// rows.  Measured with 4 heads on each of 8 KV heads, tcgen05's time over mma.sync's at 12 and 16 rows:
//  * 64 and 128 values, 1 to 64 sequences of 200 to 40,000 tokens: 0.6 to 1.4 for bf16, but 0.9 to 2.1 for q8_0 and q4_0;
//  * 256 values, 1 to 40 sequences of 300 to 12,000: 0.4 to 1.1 for bf16, but 0.7 to 1.75 for q8_0 and q4_0.
// So the threshold is where mma.sync's row tiles end, but for bf16 at 256 values, where it is where its first one does.  More
// row tiles were built and taken out again: four of them at 24 and 32 rows took longer than tcgen05 but for 64 sequences of up to
// 1500 tokens, and for 256 values, in turns of 16 rows over the same pages, the longer the more rows (64 rows: 2 to 2.5 times).
template <int FMT, int D> constexpr int kAttnTcRows = FMT == BQG_BF16 && D == 256 ? 9 : 17;

inline void attn_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, dim3 grid, int threads, int smem, cudaStream_t s,
                        bool pdl)
{
    cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
}

// CTAs of a kernel that are resident together on this device: looked up once.
template <typename K> cudaError_t attn_ctas(K kern, int threads, int smem, int *ctas)
{
    static std::mutex mu;
    static int known[64];      // per instantiation of this template: see the tag types below
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev] == 0) {
        int sms = 0, n = 0;
        if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) return e;
        if (cudaError_t e = cudaFuncSetAttribute(kern.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
        if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern.fn, threads, smem)) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        known[dev] = std::min(sms * n, kern.most);
    }
    *ctas = known[dev];
    return cudaSuccess;
}

// Units of `tile` tokens x `rows` rows that the call's arguments allow at most.
inline double attn_most(const AttnParams &p, int tile, int rows)
{
    const int64_t cap = std::min<int64_t>(p.max_pages << p.cache.lp, 0x7fff0000);
    const int64_t row_tiles = ((int64_t)p.max_q * p.group + rows - 1) / rows;
    return (double)p.n_seq * p.cache.n_kv * (double)row_tiles * (double)((cap + tile - 1) / tile);
}

// mma.sync kernel: plans the call (plan) or, plan null, launches it.
template <int FMT, int D, int RT, typename P>
cudaError_t attn_rows_call(P p, int *error, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    using G = AttnGeom<FMT, D, RT>;
    struct Kern {
        void (*fn)(const P, int *) = attn_kernel<FMT, D, RT, P>;
        int most = kAttnMaxCtas;
    } kern;
    int ctas = 0;
    if (cudaError_t e = attn_ctas(kern, 32 * kAttnWarps, G::SMEM, &ctas)) return e;
    if (plan) {
        plan->ws_bytes = kAttnHead + (size_t)2 * ctas * G::ROWS * (D + 2) * sizeof(float);
        return cudaSuccess;
    }
    p.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.counters) + kAttnHead);
    const unsigned grid = (unsigned)std::max(1.0, std::min((double)ctas, attn_most(p, kUnit, G::ROWS)));
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    attn_config(cfg, attr, dim3(grid), 32 * kAttnWarps, G::SMEM, s, pdl);
    return cudaLaunchKernelEx(&cfg, kern.fn, p, error);
}

// tcgen05 kernel and its join.
template <int FMT, int D, typename P> cudaError_t attn_tc_call(P p, int *error, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    using G = TcGeom<FMT, D>;
    struct Kern {
        void (*fn)(const P, const CUtensorMap, const CUtensorMap, int *) = attn_tc_kernel<FMT, D, P>;
        int most = (int)(kAttnSetBytes / sizeof(TcSet));
    } kern;
    int ctas = 0;
    if (cudaError_t e = attn_ctas(kern, G::THREADS, G::SMEM, &ctas)) return e;
    if (plan) {
        plan->ws_bytes = kAttnHead + (size_t)2 * ctas * G::ROWS * (D + 2) * sizeof(float);
        return cudaSuccess;
    }
    // the cache as rows of D bf16 values: boxes of 64 values x the tokens of a page (at most a tile)
    CUtensorMap kmap{}, vmap{};
    if (FMT == BQG_BF16) {
        auto enc = tensor_map_encoder();
        if (!enc) return cudaErrorNotSupported;
        const int64_t rows = (p.cache.n_pages * p.cache.n_kv) << p.cache.lp;
        if (rows > 0x7fffffff) return cudaErrorInvalidValue;        // beyond any GPU's memory at 128 bytes a row
        const cuuint64_t dim[2] = {(cuuint64_t)D, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)D * 2};
        const cuuint32_t box[2] = {64, (cuuint32_t)std::min(1 << p.cache.lp, G::TT)}, one[2] = {1, 1};
        for (int i = 0; i < 2; i++)
            if (enc(i ? &vmap : &kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, i ? p.cache.v : p.cache.k, dim, stride, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorInvalidValue;
    }
    uint8_t *ws = reinterpret_cast<uint8_t *>(p.counters);
    p.counters = reinterpret_cast<int *>(ws + kAttnCounterBytes);
    p.part = reinterpret_cast<float *>(ws + kAttnHead);
    const int grid = (int)std::max(1.0, std::min((double)ctas, attn_most(p, G::TT, kTcHalf)));
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    attn_config(cfg, attr, dim3(grid), G::THREADS, G::SMEM, s, pdl);
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern.fn, p, kmap, vmap, error)) return e;
    if (grid == 1) return cudaSuccess;                              // nothing is shared
    // the join may be set up while the first kernel runs: it waits for it before it reads
    const int rows = (int)std::min<int64_t>(G::ROWS, (int64_t)p.max_q * p.group);
    attn_config(cfg, attr, dim3(grid, (rows + 31) / 32), 256, 0, s, true);
    return cudaLaunchKernelEx(&cfg, attn_tc_join_kernel<D, G::ROWS, P>, p, grid);
}

template <int FMT, int D, typename P> cudaError_t attn_pick(const P &p, int64_t rows, int *error, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    if (rows <= 8) return attn_rows_call<FMT, D, 1, P>(p, error, plan, s, pdl);
    if constexpr (kAttnTcRows<FMT, D> > 9)
        if (rows < kAttnTcRows<FMT, D>) return attn_rows_call<FMT, D, 2, P>(p, error, plan, s, pdl);
    return attn_tc_call<FMT, D, P>(p, error, plan, s, pdl);
}

// Own tokens, a piece per warp (bqg_own.cuh).
template <int FMT, int D, int RT> cudaError_t own_call(SharedParams p, int *error, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    using G = OwnGeom<FMT, D, RT>;
    struct Kern {
        void (*fn)(const SharedParams, int *) = own_kernel<FMT, D, RT>;
        int most = kAttnMaxCtas / kAttnWarps;
    } kern;
    int ctas = 0;
    if (cudaError_t e = attn_ctas(kern, 32 * kAttnWarps, G::SMEM, &ctas)) return e;
    if (plan) {
        plan->ws_bytes = kAttnHead + (size_t)2 * ctas * kAttnWarps * G::ROWS * (D + 2) * sizeof(float);
        return cudaSuccess;
    }
    p.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.counters) + kAttnHead);
    const unsigned grid = (unsigned)std::max(1.0, std::min((double)ctas, attn_most(p, kStrip, G::ROWS)));
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    attn_config(cfg, attr, dim3(grid), 32 * kAttnWarps, G::SMEM, s, pdl);
    return cudaLaunchKernelEx(&cfg, kern.fn, p, error);
}
// Up to two row tiles (256 values: one), as the queries are held in registers; more rows go to tcgen05.  At 32 rows, 96 sequences of
// 400 tokens, 8 heads on each of 8, bf16, two sets of 16 rows over the same tokens took as long as tcgen05 (75 us).
template <int FMT, int D> cudaError_t own_pick(const SharedParams &p, int64_t rows, int *error, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    if (rows <= 8) return own_call<FMT, D, 1>(p, error, plan, s, pdl);
    if constexpr (D < 256)
        if (rows <= 16) return own_call<FMT, D, 2>(p, error, plan, s, pdl);
    return attn_tc_call<FMT, D, SharedParams>(p, error, plan, s, pdl);
}

// Shared tokens, then own ones (SharedParams).  Workspace: as for one pass, then the first one's rows.
template <int FMT, int D>
cudaError_t shared_call(SharedParams p, int *error, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    SharedParams pre = p;
    pre.own = 0;
    pre.n_seq = p.n_prefix;
    pre.max_q = (int)p.max_shared;
    p.own = 1;
    const int64_t rows = (int64_t)p.max_q * p.group, shared = p.max_shared * p.group;
    // room for every kernel that as many rows or fewer go to: a workspace for more serves fewer
    size_t at = 0;
    for (const int64_t r : {(int64_t)1, (int64_t)9, (int64_t)17}) {
        AttnPlan a{}, b{};
        if (r <= shared)
            if (cudaError_t e = attn_pick<FMT, D>(pre, r, error, &a, s, pdl)) return e;
        if (r <= rows)
            if (cudaError_t e = own_pick<FMT, D>(p, r, error, &b, s, pdl)) return e;
        at = std::max({at, a.ws_bytes, b.ws_bytes});
    }
    at = (at + 255) & ~(size_t)255;
    const size_t all = ((size_t)p.n_tokens * p.n_q + 31) & ~(size_t)31;
    if (plan) {
        plan->ws_bytes = at + all * (D + 2) * sizeof(float);
        return cudaSuccess;
    }
    pre.rows = p.rows = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.counters) + at);
    pre.rows_ml = p.rows_ml = p.rows + all * D;
    if (cudaError_t e = attn_pick<FMT, D>(pre, shared, error, nullptr, s, pdl)) return e;
    // the second pass may be set up while the first runs: it waits for it before it reads
    return own_pick<FMT, D>(p, rows, error, nullptr, s, true);
}
template <int FMT> cudaError_t shared_launch(const SharedParams &p, int D, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    int *error = nullptr;
    if (!plan)
        if (cudaError_t e = device_error_word(&error)) return e;
    if (D == 64) return shared_call<FMT, 64>(p, error, plan, s, pdl);
    if (D == 128) return shared_call<FMT, 128>(p, error, plan, s, pdl);
    return shared_call<FMT, 256>(p, error, plan, s, pdl);
}

// rows: the most rows (new tokens x heads of a group) of any sequence.
template <int FMT>
cudaError_t attn_launch(const AttnParams &p, int D, int rows, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    int *error = nullptr;
    if (!plan)
        if (cudaError_t e = device_error_word(&error)) return e;
    if (D == 64) return attn_pick<FMT, 64>(p, rows, error, plan, s, pdl);
    if (D == 128) return attn_pick<FMT, 128>(p, rows, error, plan, s, pdl);
    return attn_pick<FMT, 256>(p, rows, error, plan, s, pdl);
}

}  // namespace bqg
