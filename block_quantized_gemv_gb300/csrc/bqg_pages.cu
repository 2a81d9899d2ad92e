// bqg_pages.cu -- the accepted path of drafted tokens moved behind the context, and sequences branched.
//
// Both copy cached rows as they lie, codes and scales: no rounding, whatever the format.
//
// compact_kernel: the k-th accepted token of a sequence goes from place ctx + a_k to ctx + k; a ascends, so k <= a_k.  A
// place may be one token's source and another's goal, so the rows of one head are all read before any is written: a
// CTA takes all rows of a few heads at once, a chunk of up to 16 bytes per thread and turn, all loads before a barrier, all stores
// behind it.  Tokens that are where they belong are neither read nor written.
//
// fork_kernel: a branch gets its parent's table entries of full pages, and the tokens of its page in use, one run of
// bytes per head and side: a run per warp, four chunks per lane in flight.
#include <algorithm>

#include "bqg_pages.cuh"

namespace bqg {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxMoves = 64;

// Sides of a cache: keys, values (2 n_kv rows of heads).
template <int FMT, int D> struct Sides {
    static constexpr int RB = KvRow<FMT, D>::BYTES;
    static constexpr int SB = FMT == BQG_BF16 ? 0 : D / QK * 2;        // scales of a row: 4, 8 or 16 bytes
    static constexpr int CODES = RB / 16;                              // chunks of a row, then one of scales
    static constexpr int CHUNKS = CODES + (SB ? 1 : 0);
    static __device__ __forceinline__ uint8_t *codes(const KvCacheDev &c, int v) { return v ? c.v : c.k; }
    static __device__ __forceinline__ uint8_t *scales(const KvCacheDev &c, int v) { return reinterpret_cast<uint8_t *>(v ? c.v_scale : c.k_scale); }
    static __device__ __forceinline__ uint8_t *at(const KvCacheDev &c, int v, int64_t row, int chunk)
    {
        return chunk < CODES ? codes(c, v) + row * RB + chunk * 16 : scales(c, v) + row * SB;
    }
    static __device__ __forceinline__ uint4 load(const uint8_t *p, bool scale)
    {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (SB == 4 && scale) r.x = *reinterpret_cast<const uint32_t *>(p);
        else if (SB == 8 && scale) { const uint2 q = *reinterpret_cast<const uint2 *>(p); r.x = q.x; r.y = q.y; }
        else r = *reinterpret_cast<const uint4 *>(p);
        return r;
    }
    static __device__ __forceinline__ void store(uint8_t *p, bool scale, const uint4 &r)
    {
        if (SB == 4 && scale) *reinterpret_cast<uint32_t *>(p) = r.x;
        else if (SB == 8 && scale) *reinterpret_cast<uint2 *>(p) = make_uint2(r.x, r.y);
        else *reinterpret_cast<uint4 *>(p) = r;
    }
};

// What a sequence keeps of its path, by one warp: places lane and 32 + lane of it, good while they ascend and lie in the sequence's
// pages; how many are; its length made to fit; BQG_DEVERR_LENGTH.
struct Path { int a[2], kept, bad; int64_t ctx; };
__device__ __forceinline__ Path path_of(const CompactParams &p, int b, int lane)
{
    Path r;
    const int64_t cap = min((int64_t)0x7fff0000, p.max_pages << p.cache.lp);
    const int said = p.n_path[b], n = min(max(said, 0), p.max_q), c = p.ctx_len[b];
    r.ctx = min(max((int64_t)c, (int64_t)0), cap);
    const int32_t *path = p.path + (int64_t)b * p.max_q;
    bool good[2];
#pragma unroll
    for (int j = 0; j < 2; j++) r.a[j] = lane + 32 * j < n ? path[lane + 32 * j] : -1;
    const int low_last = __shfl_sync(0xffffffffu, r.a[0], 31);
#pragma unroll
    for (int j = 0; j < 2; j++) {
        int before = __shfl_up_sync(0xffffffffu, r.a[j], 1);
        if (lane == 0) before = j ? low_last : -1;
        good[j] = lane + 32 * j < n && r.a[j] > before && r.ctx + r.a[j] < cap;
    }
    const unsigned long long ok = (unsigned long long)__ballot_sync(0xffffffffu, good[0]) |
                                  (unsigned long long)__ballot_sync(0xffffffffu, good[1]) << 32;
    r.kept = ~ok ? __ffsll(~ok) - 1 : 64;                     // up to the first that is not
    r.bad = n != said || r.kept != n || r.ctx != c ? BQG_DEVERR_LENGTH : 0;
    return r;
}

template <int FMT, int D> __global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p)
{
    using S = Sides<FMT, D>;
    constexpr int N = (kMaxMoves * S::CHUNKS + kThreads - 1) / kThreads < 4 ? 4 : (kMaxMoves * S::CHUNKS + kThreads - 1) / kThreads;
    __shared__ int64_t from[kMaxMoves], to[kMaxMoves];        // rows of head 0
    __shared__ int n_moves;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    pdl_wait();
    pdl_launch_dependents();
    const int P = 1 << p.cache.lp;
    if (tid < 32) {
        const Path path = path_of(p, b, lane);
        const int64_t ctx = path.ctx;
        int bad = path.bad, moves = 0;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int k = lane + 32 * j;
            int64_t src = -1, dst = -1;
            bool move = k < path.kept && path.a[j] != k;
            if (move) {
                const int64_t x = ctx + path.a[j], y = ctx + k;
                const int32_t *row = p.table + (int64_t)b * p.max_pages;
                const int px = row[x >> p.cache.lp], py = row[y >> p.cache.lp];
                if (px < 0 || px >= p.cache.n_pages || py < 0 || py >= p.cache.n_pages) {
                    bad |= BQG_DEVERR_PAGE;
                    move = false;
                } else {
                    src = kv_row(p.cache, ((int64_t)px << p.cache.lp) + (x & (P - 1)), 0);
                    dst = kv_row(p.cache, ((int64_t)py << p.cache.lp) + (y & (P - 1)), 0);
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, move);
            const int at = moves + __popc(m & ((1u << lane) - 1));
            if (move) { from[at] = src; to[at] = dst; }
            moves += __popc(m);
        }
        if (slice == 0 && bad) atomicOr(p.error, bad);
        if (lane == 0) {
            n_moves = moves;
            if (slice == 0 && p.ctx_out) p.ctx_out[b] = (int)ctx + path.kept;
        }
    }
    __syncthreads();
    const int moves = n_moves, each = moves * S::CHUNKS;
    if (!moves) return;
    const int heads = 2 * p.cache.n_kv, per = (heads + p.slices - 1) / p.slices;
    const int h0 = slice * per, h1 = min(h0 + per, heads), turn = max(1, N * kThreads / each);   // heads at a time
    for (int h = h0; h < h1; h += turn) {
        const int all = min(turn, h1 - h) * each;
        uint4 r[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int x = tid + i * kThreads;
            if (x < all) {
                const int hh = h + x / each, y = x % each, c = y % S::CHUNKS;
                const bool v = hh >= p.cache.n_kv;
                const int64_t row = from[y / S::CHUNKS] + ((int64_t)(v ? hh - p.cache.n_kv : hh) << p.cache.lp);
                r[i] = S::load(S::at(p.cache, v, row, c), c >= S::CODES);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int x = tid + i * kThreads;
            if (x < all) {
                const int hh = h + x / each, y = x % each, c = y % S::CHUNKS;
                const bool v = hh >= p.cache.n_kv;
                const int64_t row = to[y / S::CHUNKS] + ((int64_t)(v ? hh - p.cache.n_kv : hh) << p.cache.lp);
                S::store(S::at(p.cache, v, row, c), c >= S::CODES, r[i]);
            }
        }
    }
}

// The new lengths alone, a warp per sequence.
__global__ void __launch_bounds__(kThreads) lengths_kernel(const CompactParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t b = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (b >= p.n_seq) return;
    const Path path = path_of(p, (int)b, threadIdx.x & 31);
    if ((threadIdx.x & 31) == 0) p.ctx_out[b] = (int)path.ctx + path.kept;
}

// `bytes` (a multiple of 4, both sides 16-byte aligned) by one warp.
__device__ __forceinline__ void warp_copy(uint8_t *dst, const uint8_t *src, int bytes, int lane)
{
    constexpr int U = 4;
    const int n = bytes / 16;
    for (int i0 = 0; i0 < n; i0 += 32 * U) {
        uint4 r[U];
#pragma unroll
        for (int i = 0; i < U; i++)
            if (i0 + 32 * i + lane < n) r[i] = *reinterpret_cast<const uint4 *>(src + (i0 + 32 * i + lane) * 16);
#pragma unroll
        for (int i = 0; i < U; i++)
            if (i0 + 32 * i + lane < n) *reinterpret_cast<uint4 *>(dst + (i0 + 32 * i + lane) * 16) = r[i];
    }
    const int rest = n * 16 + lane * 4;
    if (lane < 4 && rest < bytes) *reinterpret_cast<uint32_t *>(dst + rest) = *reinterpret_cast<const uint32_t *>(src + rest);
}

template <int FMT, int D> __global__ void __launch_bounds__(kThreads) fork_kernel(const ForkParams p)
{
    using S = Sides<FMT, D>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int i = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    pdl_wait();
    pdl_launch_dependents();
    const int up = p.parent[i], child = p.child[i], fresh = p.fresh[i];
    if (up < 0 || up >= p.n_rows || child < 0 || child >= p.n_rows || up == child) {
        if (slice == 0 && tid == 0) atomicOr(p.error, BQG_DEVERR_ROW);
        return;
    }
    const int64_t cap = min((int64_t)0x7fff0000, p.max_pages << p.cache.lp);
    const int said = p.ctx_len[up];
    const int ctx = (int)min(max((int64_t)said, (int64_t)0), cap);
    const int64_t full = ctx >> p.cache.lp;
    const int used = ctx & ((1 << p.cache.lp) - 1);
    const int32_t *from = p.table + (int64_t)up * p.max_pages;
    int32_t *to = p.table + (int64_t)child * p.max_pages;
    int bad = said != ctx ? BQG_DEVERR_LENGTH : 0;
    if (slice == 0) {
        for (int64_t x = tid; x < full; x += kThreads) to[x] = from[x];
        if (tid == 0) {
            if (full < p.max_pages) to[full] = fresh;
            p.ctx_len[child] = ctx;
        }
    }
    if (used) {
        const int old = from[full];
        if (old < 0 || old >= p.cache.n_pages || fresh < 0 || fresh >= p.cache.n_pages) {
            bad |= BQG_DEVERR_PAGE;
        } else if (old != fresh) {
            for (int h = slice * kWarps + warp; h < 2 * p.cache.n_kv; h += p.slices * kWarps) {
                const bool v = h >= p.cache.n_kv;
                const int head = v ? h - p.cache.n_kv : h;
                const int64_t a = kv_row(p.cache, (int64_t)old << p.cache.lp, head), b = kv_row(p.cache, (int64_t)fresh << p.cache.lp, head);
                warp_copy(S::codes(p.cache, v) + b * S::RB, S::codes(p.cache, v) + a * S::RB, used * S::RB, lane);
                if constexpr (S::SB > 0)
                    warp_copy(S::scales(p.cache, v) + b * S::SB, S::scales(p.cache, v) + a * S::SB, used * S::SB, lane);
            }
        }
    }
    if (slice == 0 && tid == 0 && bad) atomicOr(p.error, bad);
}

template <typename P> cudaError_t launch(void (*kern)(P), const P &p, int64_t ctas, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}
template <int FMT> void (*compact_fn(int D))(CompactParams)
{
    return D == 64 ? compact_kernel<FMT, 64> : D == 128 ? compact_kernel<FMT, 128> : compact_kernel<FMT, 256>;
}
template <int FMT> void (*fork_fn(int D))(ForkParams)
{
    return D == 64 ? fork_kernel<FMT, 64> : D == 128 ? fork_kernel<FMT, 128> : fork_kernel<FMT, 256>;
}

}  // namespace

cudaError_t launch_compact(CompactParams p, int fmt, int D, int sms, cudaStream_t s, bool pdl)
{
    if (cudaError_t e = device_error_word(&p.error)) return e;
    // six CTAs per SM, if there are heads for them (resident together but for bf16 of 256 values, where registers let four be)
    p.slices = (int)std::min<int64_t>(2 * p.cache.n_kv, std::max<int64_t>(1, (int64_t)sms * 6 / p.n_seq));
    auto fn = fmt == BQG_Q8_0 ? compact_fn<BQG_Q8_0>(D) : fmt == BQG_Q4_0 ? compact_fn<BQG_Q4_0>(D) : compact_fn<BQG_BF16>(D);
    int32_t *const apart = p.ctx_in_table ? p.ctx_out : nullptr;
    if (apart) p.ctx_out = nullptr;
    if (cudaError_t e = launch(fn, p, (int64_t)p.n_seq * p.slices, s, pdl)) return e;
    if (!apart) return cudaSuccess;
    p.ctx_out = apart;                                        // behind all reads of the table
    return launch(lengths_kernel, p, ((int64_t)p.n_seq + kWarps - 1) / kWarps, s, pdl);
}

cudaError_t launch_fork(ForkParams p, int fmt, int D, int sms, cudaStream_t s, bool pdl)
{
    if (cudaError_t e = device_error_word(&p.error)) return e;
    // eight CTAs per SM, if there are runs for them (five are resident for bf16, three for codes: 48 and 75 to 80 registers)
    const int runs = (2 * p.cache.n_kv + kWarps - 1) / kWarps;
    p.slices = (int)std::min<int64_t>(runs, std::max<int64_t>(1, (int64_t)sms * 8 / p.n));
    auto fn = fmt == BQG_Q8_0 ? fork_fn<BQG_Q8_0>(D) : fmt == BQG_Q4_0 ? fork_fn<BQG_Q4_0>(D) : fork_fn<BQG_BF16>(D);
    return launch(fn, p, (int64_t)p.n * p.slices, s, pdl);
}

}  // namespace bqg
