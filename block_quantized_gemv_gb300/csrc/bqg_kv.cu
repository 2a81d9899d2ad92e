// bqg_kv.cu -- per-head norm and rotation of queries and keys, the cache's
// encoder and decoder.
//
// norm_rope_kernel: one warp per head row of one token (queries, keys and
// values of a token are consecutive rows).  Lane l holds the E = D / 32
// values from E l on, so a row is one load of 4 to 32 bytes per lane, its
// sum of squares one warp reduction, and a 32-value block sits in 32 / E
// neighbouring lanes.  A pair (i, i + R/2) is R/2/E lanes apart (R is a
// multiple of 16, E divides 8): one exchange; an adjacent pair is in one lane.
// Everything is fp32 with the roundings of include/bqgemv.h; the sum of
// squares is kept as error-free fp32 pairs (SumSq), so r matches the fp64
// definition up to a rare tie.
#include <algorithm>

#include "bqg_kv.cuh"

namespace bqg {

// Bits of out-of-range indices met (BQG_DEVERR_*).
__device__ int g_kv_error;

cudaError_t kv_take_error(int *out)
{
    int v = 0, zero = 0;
    if (cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(int))) return e;
    if (v)
        if (cudaError_t e = cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(int))) return e;
    *out = v;
    return cudaSuccess;
}

namespace {

constexpr int kWarps = 8;      // warps per CTA

template <int E> __device__ __forceinline__ void load_row(const void *x, int x_f32, int64_t first, float (&v)[E])
{
    if (x_f32) {
        const float *p = reinterpret_cast<const float *>(x) + first;
        if constexpr (E == 2) {
            const float2 a = *reinterpret_cast<const float2 *>(p);
            v[0] = a.x; v[1] = a.y;
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(p + i);
                v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
            }
        }
    } else {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(x) + first;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(p + i);
            v[i] = bf16_lo(w); v[i + 1] = bf16_hi(w);
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int E> __device__ __forceinline__ void store_bf16(uint16_t *p, const float (&v)[E])
{
    if constexpr (E == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16x2_rn(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            *reinterpret_cast<uint2 *>(p + i) =
                make_uint2(pack_bf16x2_rn(v[i], v[i + 1]), pack_bf16x2_rn(v[i + 2], v[i + 3]));
    }
}

// r = fp32(1 / sqrt(sum x^2 / D + eps)) of the row held by the warp.
template <int E> __device__ __forceinline__ float row_rms_recip(const float (&x)[E], float eps)
{
    SumSq acc;
#pragma unroll
    for (int i = 0; i < E; i++) acc.add(x[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        acc.merge(__shfl_xor_sync(0xffffffffu, acc.hi, o), __shfl_xor_sync(0xffffffffu, acc.lo, o));
    const bool wide = __any_sync(0xffffffffu, acc.wide != 0.0);
    // every lane holds the same pair up to the order of the sums: take lane 0's
    const float hi = __shfl_sync(0xffffffffu, acc.hi, 0), lo = __shfl_sync(0xffffffffu, acc.lo, 0);
    if (!wide && hi >= 0x1p-60f && hi <= 0x1p100f) return rms_recip_pair(hi, lo, (float)(E * 32), eps);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc.wide += __shfl_xor_sync(0xffffffffu, acc.wide, o);
    const double t = ((double)hi + (double)lo) + __shfl_sync(0xffffffffu, acc.wide, 0);
    return (float)(1.0 / sqrt(t / (double)(E * 32) + (double)eps));
}

// The warp's row (E values per lane) into cache row `row`.
template <int FMT, int D>
__device__ __forceinline__ void encode_row(const float (&y)[D / 32], int lane, uint8_t *codes, uint16_t *scales, int64_t row)
{
    constexpr int E = D / 32, LB = 32 / E;            // lanes per block
    uint8_t *dst = codes + row * KvRow<FMT, D>::BYTES;
    if constexpr (FMT == BQG_BF16) {
        store_bf16<E>(reinterpret_cast<uint16_t *>(dst) + lane * E, y);
    } else if constexpr (FMT == BQG_Q8_0) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < E; i++) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
        for (int o = LB / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const __half dh = __float2half_rn(__fdiv_rn(amax, 127.0f));
        const float d = __half2float(dh);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const uint32_t a = (uint8_t)(int8_t)q8_code(y[i], d), b = (uint8_t)(int8_t)q8_code(y[i + 1], d);
            *reinterpret_cast<uint16_t *>(dst + lane * E + i) = (uint16_t)(a | (b << 8));
        }
        if (lane % LB == 0) scales[row * KvRow<FMT, D>::NB + lane / LB] = __half_as_ushort(dh);
    } else {
        // signed value of largest magnitude, the first one on ties
        float bv = y[0], ba = fabsf(y[0]);
#pragma unroll
        for (int i = 1; i < E; i++)
            if (fabsf(y[i]) > ba) { bv = y[i]; ba = fabsf(y[i]); }
        int bl = lane;
#pragma unroll
        for (int o = LB / 2; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const float oa = __shfl_xor_sync(0xffffffffu, ba, o);
            const int ol = __shfl_xor_sync(0xffffffffu, bl, o);
            if (oa > ba || (oa == ba && ol < bl)) { bv = ov; ba = oa; bl = ol; }
        }
        const __half dh = __float2half_rn(__fdiv_rn(bv, -8.0f));
        const float d = __half2float(dh);
        uint32_t q[E];
#pragma unroll
        for (int i = 0; i < E; i++) {
            q[i] = 8;
            if (d != 0.0f) q[i] = (uint32_t)fminf(fmaxf(roundf(__fdiv_rn(y[i], d)) + 8.0f, 0.0f), 15.0f);
            q[i] |= __shfl_xor_sync(0xffffffffu, q[i], LB / 2) << 4;      // lower half: the value 16 further on
        }
        if (lane % LB < LB / 2) {
            const int at = (lane / LB) * 16 + (lane % LB) * E;
#pragma unroll
            for (int i = 0; i < E; i += 2)
                *reinterpret_cast<uint16_t *>(dst + at + i) = (uint16_t)((q[i] & 0xffu) | ((q[i + 1] & 0xffu) << 8));
        }
        if (lane % LB == 0) scales[row * KvRow<FMT, D>::NB + lane / LB] = __half_as_ushort(dh);
    }
}

template <int FMT, int D> __global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormRopeParams p)
{
    constexpr int E = D / 32;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int rows = p.n_q + (p.k ? p.n_kv : 0) + (p.v ? p.n_kv : 0);       // rows of one token
    for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < p.T * rows;
         i += (int64_t)gridDim.x * kWarps) {
        const int64_t t = i / rows;
        int h = (int)(i - t * rows);
        const int what = h < p.n_q ? 0 : (p.k && h < p.n_q + p.n_kv) ? 1 : 2;       // query, key, value
        h -= what == 0 ? 0 : what == 1 ? p.n_q : rows - p.n_kv;
        int64_t slot = -1;
        if (what && p.slots) {
            slot = p.slots[t];
            if (slot >= 0 && !kv_slot_ok(p.cache, slot)) {
                if (lane == 0) atomicOr(&g_kv_error, BQG_DEVERR_SLOT);
                slot = -1;
            }
            if (slot < 0) continue;
        }
        float y[E];
        const void *x = what == 0 ? p.q : what == 1 ? p.k : p.v;
        const int64_t stride = what == 0 ? p.q_stride : what == 1 ? p.k_stride : p.v_stride;
        load_row<E>(x, p.x_f32, t * stride + (int64_t)h * D + lane * E, y);
        if (what < 2 && p.norm) {
            const float r = row_rms_recip<E>(y, p.eps);
            const float *g = what ? p.gamma_k : p.gamma_q;
#pragma unroll
            for (int j = 0; j < E; j++) {
                y[j] = __fmul_rn(y[j], r);
                if (g) y[j] = __fmul_rn(y[j], g[lane * E + j]);
            }
        }
        bool lost = false;
        if (what < 2 && p.rot) {
            const int64_t pos = p.pos[t];
            lost = pos < 0 || pos >= p.n_pos;
            if (lost && lane == 0) atomicOr(&g_kv_error, BQG_DEVERR_POSITION);
            const float *row = p.table + (lost ? 0 : pos) * p.rot;
            const int half = p.rot / 2;
            if (p.interleaved) {
                if (lane * E < p.rot) {
#pragma unroll
                    for (int j = 0; j < E; j += 2) {
                        const int pair = (lane * E + j) / 2;
                        const float c = row[pair], s = row[half + pair], a = y[j], b = y[j + 1];
                        y[j] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
                        y[j + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
                    }
                }
            } else {
                const bool low = lane * E < half, in = lane * E < p.rot;
                const int other = !in ? lane : low ? lane + half / E : lane - half / E;
#pragma unroll
                for (int j = 0; j < E; j++) {
                    const float o = __shfl_sync(0xffffffffu, y[j], other);
                    if (in) {
                        const int pair = lane * E + j - (low ? 0 : half);
                        const float c = row[pair], s = row[half + pair];
                        y[j] = low ? __fsub_rn(__fmul_rn(y[j], c), __fmul_rn(o, s))
                                   : __fadd_rn(__fmul_rn(o, s), __fmul_rn(y[j], c));
                    }
                }
            }
        }
        if (what && p.slots) {
            if (!lost)
                encode_row<FMT, D>(y, lane, what == 1 ? p.cache.k : p.cache.v,
                                   what == 1 ? p.cache.k_scale : p.cache.v_scale, kv_row(p.cache, slot, h));
        } else {
#pragma unroll
            for (int j = 0; j < E; j++) y[j] = lost ? 0.f : y[j];
            uint16_t *out = what ? p.k_out : p.q_out;
            store_bf16<E>(out + (t * (what ? p.n_kv : p.n_q) + h) * D + lane * E, y);
        }
    }
}

// Sixteen values of one cached row per thread: values 16 j .. of the row
// (bf16, q8_0), or the low and high nibbles of eight code bytes (q4_0:
// values 8 (j % 2) .. and 16 + 8 (j % 2) .. of block j / 2).
template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadParams p)
{
    constexpr int J = D / 16;                           // threads per row
    pdl_wait();
    pdl_launch_dependents();
    const int n_kv = p.cache.n_kv;
    const int64_t per = p.T * n_kv * J, stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < 2 * per; i += stride) {
        const bool is_v = i >= per;
        const int64_t rest = is_v ? i - per : i;
        const int64_t t = rest / (n_kv * J);
        const int hj = (int)(rest - t * (n_kv * J)), h = hj / J, j = hj % J;
        int64_t slot = p.slots[t];
        if (slot >= 0 && !kv_slot_ok(p.cache, slot)) {
            atomicOr(&g_kv_error, BQG_DEVERR_SLOT);
            slot = -1;
        }
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; e++) f[e] = 0.f;
        if (slot >= 0) {
            const int64_t row = kv_row(p.cache, slot, h);
            const uint8_t *src = (is_v ? p.cache.v : p.cache.k) + row * KvRow<FMT, D>::BYTES;
            if constexpr (FMT == BQG_BF16) {
                const uint4 a = *reinterpret_cast<const uint4 *>(src + 32 * j);
                const uint4 b = *reinterpret_cast<const uint4 *>(src + 32 * j + 16);
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int e = 0; e < 8; e++) { f[2 * e] = bf16_lo(w[e]); f[2 * e + 1] = bf16_hi(w[e]); }
            } else {
                const float d = half_bits_to_float((is_v ? p.cache.v_scale : p.cache.k_scale)[row * (D / QK) + j / 2]);
                if constexpr (FMT == BQG_Q8_0) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(src + 16 * j);
                    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int e = 0; e < 16; e++) f[e] = (float)(int8_t)(w[e / 4] >> (8 * (e % 4))) * d;   // exact
                } else {
                    const uint2 a = *reinterpret_cast<const uint2 *>(src + 8 * j);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int byte = (int)((e < 4 ? a.x : a.y) >> (8 * (e % 4))) & 0xff;
                        f[e] = (float)((byte & 15) - 8) * d;                                          // exact
                        f[8 + e] = (float)((byte >> 4) - 8) * d;
                    }
                }
            }
        }
        // first value of f[0..7] and of f[8..15] in the row
        const int lo = (FMT == BQG_Q4_0) ? 32 * (j / 2) + 8 * (j % 2) : 16 * j;
        const int hi = (FMT == BQG_Q4_0) ? lo + 16 : lo + 8;
        const int64_t o = (t * n_kv + h) * D;
        void *out = is_v ? p.v_out : p.k_out;
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const float *g = f + 8 * s;
            const int64_t at = o + (s ? hi : lo);
            if constexpr (F32) {
                float4 *dst = reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + at);
                dst[0] = make_float4(g[0], g[1], g[2], g[3]);
                dst[1] = make_float4(g[4], g[5], g[6], g[7]);
            } else {
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + at) =
                    make_uint4(pack_bf16x2_rn(g[0], g[1]), pack_bf16x2_rn(g[2], g[3]), pack_bf16x2_rn(g[4], g[5]),
                               pack_bf16x2_rn(g[6], g[7]));
            }
        }
    }
}

template <typename P> cudaError_t launch(void (*kern)(P), const P &p, int64_t ctas, int threads, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(ctas, 0x7fffffff));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int FMT> void (*norm_rope_fn(int D))(NormRopeParams)
{
    return D == 64 ? norm_rope_kernel<FMT, 64> : D == 128 ? norm_rope_kernel<FMT, 128> : norm_rope_kernel<FMT, 256>;
}
template <int FMT, bool F32> void (*kv_read_fn(int D))(KvReadParams)
{
    return D == 64 ? kv_read_kernel<FMT, 64, F32> : D == 128 ? kv_read_kernel<FMT, 128, F32> : kv_read_kernel<FMT, 256, F32>;
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, int fmt, int D, int sms, cudaStream_t s, bool pdl)
{
    const int64_t rows = p.T * (p.n_q + (p.k ? p.n_kv : 0) + (p.v ? p.n_kv : 0));
    if (rows == 0) return cudaSuccess;
    auto fn = fmt == BQG_Q8_0 ? norm_rope_fn<BQG_Q8_0>(D) : fmt == BQG_Q4_0 ? norm_rope_fn<BQG_Q4_0>(D) : norm_rope_fn<BQG_BF16>(D);
    return launch(fn, p, std::min<int64_t>((rows + kWarps - 1) / kWarps, (int64_t)sms * 8), 32 * kWarps, s, pdl);
}

cudaError_t launch_kv_read(const KvReadParams &p, int fmt, int D, int out_f32, int sms, cudaStream_t s, bool pdl)
{
    const int64_t n = 2 * p.T * p.cache.n_kv * (D / 16);
    if (n == 0) return cudaSuccess;
    auto fn = out_f32 ? (fmt == BQG_Q8_0 ? kv_read_fn<BQG_Q8_0, true>(D) : fmt == BQG_Q4_0 ? kv_read_fn<BQG_Q4_0, true>(D) : kv_read_fn<BQG_BF16, true>(D))
                      : (fmt == BQG_Q8_0 ? kv_read_fn<BQG_Q8_0, false>(D) : fmt == BQG_Q4_0 ? kv_read_fn<BQG_Q4_0, false>(D) : kv_read_fn<BQG_BF16, false>(D));
    return launch(fn, p, std::min<int64_t>((n + 255) / 256, (int64_t)sms * 8), 256, s, pdl);
}

}  // namespace bqg
