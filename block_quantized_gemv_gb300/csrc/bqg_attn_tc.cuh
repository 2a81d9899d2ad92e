// bqg_attn_tc.cuh -- the same attention for many rows per KV head, on tcgen05.
//
// With R = new tokens x heads of a group rows sharing a KV head, the two
// products cost R multiply-adds per cached value: from a few dozen rows on the
// tensor cores and not the stream decide, and mma.sync cannot feed them.
// Here a tile is 128 rows (the MMA's M) x 128 cached tokens:
//     S = Q K^T  (N = 128 tokens, K = D),   O += P V  (N = D, K = 128 tokens)
// with Q, K and V in shared memory (128-byte swizzle; V is the N-major operand
// as it lies, tokens x values), and S, P and O in tensor memory: P takes
// the place of S, two fp16 or bf16 per column, and is the second product's A operand.
//
//  * Two streams of tiles share a CTA, each with its own S, O, maximum and
//    sum, so that one stream's softmax runs under the other's products.  With
//    more than 128 rows in a row group (up to 256) the streams are its two halves
//    over the same keys and values; with at most 128 they are the even and the odd
//    tiles of the same rows, joined at the end.
//  * Warps 0-3 and 4-7: softmax of stream 0 and 1, one row per thread: a
//    first pass over the row's 128 scores for their maximum, a second for the
//    exponentials.  The running maximum is raised only when exceeded by kSlack
//    (see bqg_attn.cuh), and only then is O rescaled, after the products so far.
//  * Warp 8: issues the products, in an order that alternates the streams.
//  * Warp 9 brings keys and values.  bf16: straight into the ring of tiles, in TMA boxes
//    of 64 values x the tokens of a page.  q8_0 / q4_0: codes and scales as they
//    lie, one bulk copy each per page, into a ring of their own, from which warps
//    10-17 build the tile: codes as fp16 integers (bqg_attn.cuh), times the
//    block's scale: one rounding (relative 2^-12, for keys too: a block's scale
//    cannot be applied behind a product that sums over all blocks).
//  * Tiles are shared out evenly over the CTAs as in bqg_attn.cuh, a tile of two
//    halves counting twice.  Sets of tiles that several CTAs share leave partial
//    results, which a second, small launch joins: with up to 256 rows of
//    them, the CTA that came last took longer for it than the whole GPU does.
//  * Every wait is bounded; one that gives up sets the error word, and the
//    rest of the CTA's work is skipped.
//
// A drafted token's infinite or NaN value must not reach rows that do not see
// it, and 0 x NaN in the product would.  In tiles that hold new tokens the
// loader stores zeros for such values and marks the piece; the rows that see the
// token add them (infinities and NaN stay what they are) when they are written.
#pragma once

#include <cuda.h>

#include "bqg_attn.cuh"
#include "bqg_tc.cuh"

namespace bqg {

constexpr int kTcTile = 128;             // tokens of a tile, rows of a stream
constexpr int kTcRows = 2 * kTcTile;     // rows of a row group
constexpr int kTcSoftmaxWarps = 8;
constexpr int kTcMmaWarp = 8, kTcCopyWarp = 9;

// A set of tiles shared by several CTAs, as its first CTA describes it for the join (rows 0: none).
struct TcSet {
    int rows, row0, h, q0;      // rows of the group, the first one; KV head; the sequence's first query token
    int c0, c1, pad0, pad1;     // CTAs
};

template <int FMT, int D> struct TcGeom {
    static constexpr bool QUANT = FMT != BQG_BF16;
    static constexpr int BUILD_WARPS = QUANT ? 8 : 0;
    static constexpr int THREADS = 32 * (kTcSoftmaxWarps + 2 + BUILD_WARPS);
    static constexpr int HALVES = D / 64;                               // 64 values: one 128-byte swizzle atom wide
    static constexpr int HALF = kTcTile * 128;                          // bytes of a tile's half
    static constexpr int TILE = HALVES * HALF;                          // one tile of Q, K or V in fp16 / bf16
    static constexpr int NS = QUANT && D == 128 ? 3 : 4;                // ring slots (see tc_k_pos)
    static constexpr int RB = KvRow<FMT, D>::BYTES;
    static constexpr int NB = D / QK;
    static constexpr int CPT = RB / 16;                                 // 16-byte chunks of a cached row
    static constexpr int NC = kTcTile * CPT / 256;                      // chunks per building thread and side
    static constexpr int RAW = QUANT ? kTcTile * (RB + 2 * NB) : 0;     // codes, then scales, of a side
    static constexpr int NR = !QUANT ? 0 : 52 * 1024 / (QUANT ? RAW : 1); // raw sides in flight: up to 52 KiB
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_RAW = OFF_RING + NS * TILE;
    static constexpr int OFF_ML = OFF_RAW + NR * RAW;                   // (maximum, sum) per stream and row
    static constexpr int OFF_BARS = OFF_ML + 2 * kTcTile * 8;
    // full, empty per slot; raw full, empty; s_full, p_full, o_done per stream; q_full; the softmax warps' meeting
    // point; values landed
    static constexpr int NBARS = 2 * NS + 2 * NR + 6 + 1 + 1 + 1;
    static constexpr int OFF_WORDS = OFF_BARS + NBARS * 8;              // TMEM base, abort, -, 4 NaN marks, 8 page marks
    static constexpr int OFF_SIDES = (OFF_WORDS + 64 + 15) / 16 * 16;   // what a raw side holds, 16 bytes each
    static constexpr int SMEM = OFF_SIDES + 16 * NR + 1024;             // + slack for 1024-byte alignment
    static constexpr int S0 = 0, O0 = 256;                              // tensor memory columns, + 128 per stream
    static_assert(SMEM <= 232448, "shared memory");
};

// Positions of tile g's keys and values in the rings' order K0 K1 V0 K2 V1 K3 V2 ..., which is the order in
// which the products take them (g counts all tiles of the CTA; the last values leave one position unused).
__device__ __forceinline__ int tc_k_pos(int g) { return g == 0 ? 0 : 2 * g - 1; }
__device__ __forceinline__ int tc_v_pos(int g) { return 2 * g + 2; }

// The pieces of one CTA: consecutive tiles of one (sequence, KV head, row group).
struct TcPiece {
    AttnSeq s;
    int h, row0, rows;          // first row of the group, its rows (at most kTcRows)
    int nq;                     // 2: the streams are two halves of the rows; 1: even and odd tiles
    int tile0, n;               // tiles of the piece
    int c0, c1;                 // CTAs that share the (sequence, KV head, row group)
};
struct TcWork {
    int64_t per, cur, end, base;
    AttnSeq s;
    __device__ static __forceinline__ int64_t cost(const AttnParams &p, const AttnSeq &q)
    {
        const int tiles = (q.len + kTcTile - 1) / kTcTile, halves = (q.T * p.group + kTcTile - 1) / kTcTile;
        return (int64_t)p.cache.n_kv * tiles * halves;
    }
    __device__ __forceinline__ void init(const AttnParams &p, int lane, int &bad)
    {
        auto weight = [&](const AttnSeq &q) { return cost(p, q); };
        const int64_t total = attn_total(p, lane, weight, bad);
        // at least two, so that every range between a set's first and last holds the beginning of a tile
        per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)2);
        cur = per * blockIdx.x;
        end = min(cur + per, total);
        base = 0;
        s = AttnSeq{};
        if (cur < end) {
            int ignored = 0;
            s = attn_seq(p, attn_find(p, cur, lane, weight, base), ignored);
        }
    }
    __device__ __forceinline__ bool next(const AttnParams &p, TcPiece &o)
    {
        int ignored = 0;
        while (cur < end) {
            while (cur - base >= cost(p, s)) {
                base += cost(p, s);
                s = attn_seq(p, s.b + 1, ignored);
            }
            const int tiles = (s.len + kTcTile - 1) / kTcTile, all = s.T * p.group;
            const int halves = (all + kTcTile - 1) / kTcTile, groups = (halves + 1) / 2;
            const int64_t off = cur - base, head = (int64_t)tiles * halves;
            o.h = (int)(off / head);
            const int64_t rem = off - o.h * head;
            const int g = min((int)(rem / (2 * tiles)), groups - 1);
            o.row0 = g * kTcRows;
            o.rows = min(kTcRows, all - o.row0);
            o.nq = o.rows > kTcTile ? 2 : 1;
            const int64_t seg = base + o.h * head + (int64_t)g * 2 * tiles;       // its first tile's number
            o.tile0 = (int)((cur - seg + o.nq - 1) / o.nq);                       // tiles that begin in this range
            const int last = (int)min((int64_t)tiles, (end - seg + o.nq - 1) / o.nq);
            o.n = last - o.tile0;
            cur = seg + (int64_t)max(last, o.tile0) * o.nq;
            if (o.n <= 0) continue;
            o.c0 = (int)(seg / per);
            o.c1 = (int)((seg + (int64_t)(tiles - 1) * o.nq) / per);
            o.s = s;
            return true;
        }
        return false;
    }
};

// N-major operand (V: tokens x values, 128-byte swizzle): 64 values x 8
// tokens per atom; the next 64 values are HALF bytes on, the next 8 tokens 1024.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t half)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3fff);
    d |= (uint64_t)(half >> 4) << 16;                  // leading byte offset: the next 64 values
    d |= (uint64_t)(1024 >> 4) << 32;                  // stride byte offset: the next 8 tokens
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// D[tmem] (+)= A[smem descriptor] * B[smem descriptor]
__device__ __forceinline__ void umma_f16_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void tma_box_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Byte offset of 16-byte chunk c (eight values) of row r in a swizzled tile.
__device__ __forceinline__ uint32_t tc_chunk(int r, int c)
{
    return (uint32_t)((c >> 3) * (kTcTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Value `dim` of cached row `row`, as far as it is an infinity or NaN; 0 otherwise.
template <int FMT, int D> __device__ float tc_nonfinite(const KvCacheDev &c, int64_t row, int dim)
{
    float f;
    if constexpr (FMT == BQG_BF16) {
        f = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(c.v)[row * D + dim] << 16);
    } else {
        const float d = half_bits_to_float(c.v_scale[row * (D / QK) + dim / QK]);
        if constexpr (FMT == BQG_Q8_0) {
            f = (float)(int8_t)c.v[row * D + dim] * d;
        } else {
            const int byte = c.v[row * (D / 2) + dim / QK * 16 + dim % 16];
            f = (float)((dim % QK < 16 ? byte & 15 : byte >> 4) - 8) * d;
        }
    }
    return isfinite(f) ? 0.f : f;
}

// Partial results of a piece: values in groups of four, [slot][D / 4][kTcRows][4] (a warp's 32 rows are then
// 512 contiguous bytes), and (maximum, sum) [slot][kTcRows].
template <int FMT, int D>
__global__ void __launch_bounds__(TcGeom<FMT, D>::THREADS, 1)
attn_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int *error)
{
    using G = TcGeom<FMT, D>;
    constexpr bool BF = (FMT == BQG_BF16);
    constexpr float NEG = -__builtin_huge_valf();
    constexpr float kShift = BF ? 0.0f : 8.0f;
    constexpr int NS = G::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bars = sb + G::OFF_BARS;
    auto bar_full = [&](int i) { return bars + 8 * i; };
    auto bar_empty = [&](int i) { return bars + 8 * (NS + i); };
    auto bar_s = [&](int s) { return bars + 8 * (2 * NS + s); };
    auto bar_p = [&](int s) { return bars + 8 * (2 * NS + 2 + s); };
    auto bar_o = [&](int s) { return bars + 8 * (2 * NS + 4 + s); };
    auto bar_rawf = [&](int i) { return bars + 8 * (2 * NS + 9 + i); };
    auto bar_rawe = [&](int i) { return bars + 8 * (2 * NS + 9 + G::NR + i); };
    const uint32_t bar_q = bars + 8 * (2 * NS + 6), bar_meet = bars + 8 * (2 * NS + 7), bar_land = bars + 8 * (2 * NS + 8);
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_WORDS);
    volatile uint32_t *const abort_flag = words + 1, *const nan_mark = words + 3;
    volatile uint8_t *const dead_strips = reinterpret_cast<volatile uint8_t *>(smem + G::OFF_WORDS + 28);   // [tile & 7]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(bar_full(i), G::QUANT ? G::BUILD_WARPS : 1);
            mbar_init(bar_empty(i), 1);                // tcgen05.commit
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(bar_s(s), 1);                    // tcgen05.commit
            mbar_init(bar_p(s), 4);                    // the stream's softmax warps
            mbar_init(bar_o(s), 1);                    // tcgen05.commit
        }
        mbar_init(bar_q, kTcSoftmaxWarps);
        mbar_init(bar_meet, kTcSoftmaxWarps);
        mbar_init(bar_land, 1);
        for (int i = 0; i < G::NR; i++) {
            mbar_init(bar_rawf(i), 1);
            mbar_init(bar_rawe(i), G::BUILD_WARPS);
        }
        for (int i = 1; i < 7; i++) words[i] = 0;
        mbar_fence_init();
    }
    if (warp == kTcMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + G::OFF_WORDS), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = words[0];
    pdl_wait();
    pdl_launch_dependents();

    auto fail = [&]() {
        if (!*abort_flag) atomicOr(error, 2);
        *abort_flag = 1;
    };
    int bad = 0;
    TcWork work;
    work.init(p, lane, bad);
    if (bad && blockIdx.x == 0 && warp == 0) atomicOr(error, bad);
    TcPiece w;

    if (warp < kTcSoftmaxWarps) {
        // ---------------- softmax and results ----------------
        const int st = warp >> 2, r = (warp & 3) * 32 + lane;                // stream, row of its tile
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lanes + G::S0 + 128 * st, to = lanes + G::O0 + 128 * st;
        float *const ml = reinterpret_cast<float *>(smem + G::OFF_ML);
        float *const part_ml = p.part + (int64_t)2 * gridDim.x * kTcRows * D;
        TcSet set{};                                                         // begun here, ended elsewhere
        int jobs = 0, pieces = 0, meets = 0, tiles_seen = 0;
        bool ok = true;
        // all softmax warps; false once a wait has given up anywhere
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_meet);
            ok = __all_sync(0xffffffffu, mbar_wait_spin(bar_meet, meets & 1));
            meets++;
            if (!ok) fail();
            return ok;
        };
        while (ok && work.next(p, w)) {
            const int grow = w.nq == 2 ? st * kTcTile + r : r;               // row of the group
            const bool row_ok = grow < w.rows;
            const bool warp_ok = __any_sync(0xffffffffu, row_ok);
            // the row's query into shared memory, and its softmax scale
            const uint16_t *src = row_ok ? attn_q_row(p, w.s, w.h, w.row0 + grow, D) : nullptr;
            float rs = p.scale_log2, inv = 1.f;
            if constexpr (!BF) {
                float top = 0.f;
                if (src)
#pragma unroll 4
                    for (int c = 0; c < D / 8; c++) {
                        float f[8];
                        bf16x8_to_f32(*reinterpret_cast<const uint4 *>(src + 8 * c), f);
#pragma unroll
                        for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(f[i]));
                    }
                if (top > 0.f && top < __int_as_float(0x7f800000)) {
                    const uint32_t ex = min(__float_as_uint(top) >> 23, 253u);
                    inv = __uint_as_float((254u - ex) << 23);
                    rs = fmaxf(p.scale_log2 * (1.0f / inv), 1.17549435e-38f);
                }
            }
            if (st == 0 || w.nq == 2) {
                const uint32_t dst = sb + G::OFF_Q + st * G::TILE;
#pragma unroll 4
                for (int c = 0; c < D / 8; c++) {
                    uint4 v = src ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0, 0, 0, 0);
                    if constexpr (!BF) {
                        float f[8];
                        bf16x8_to_f32(v, f);
                        v = make_uint4(pack2<false>(f[0] * inv, f[1] * inv), pack2<false>(f[2] * inv, f[3] * inv),
                                       pack2<false>(f[4] * inv, f[5] * inv), pack2<false>(f[6] * inv, f[7] * inv));
                    }
                    sts128(dst + tc_chunk(r, c), v);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_q);
            const unsigned long long sees = row_ok ? attn_sees(p, w.s, w.row0 + grow) : 0;

            float top = NEG, sum = 0.f;
            bool first = true;
            for (int i = (w.nq == 2 ? 0 : st); i < w.n; i += 3 - w.nq) {
                const bool ready = mbar_wait_spin(bar_s(st), jobs & 1);
                if (!__all_sync(0xffffffffu, ready) || *abort_flag) { fail(); ok = false; break; }
                tc_fence_after();
                const int tok0 = (w.tile0 + i) * kTcTile;
                const unsigned dead = dead_strips[(tiles_seen + i) & 7];
                const bool edge = tok0 + kTcTile > w.s.ctx || dead;
                if (warp_ok) {
                    uint32_t live[4];                                        // tokens that this row sees, 32 per word
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < 4; c++) {
                            const int t0 = tok0 + 32 * c, before = w.s.ctx - t0, all = w.s.len - t0;
                            uint32_t m = before >= 32 ? ~0u : before > 0 ? (1u << before) - 1 : 0u;
                            if (before < 32) m |= before > 0 ? (uint32_t)sees << before : -before < 64 ? (uint32_t)(sees >> -before) : 0u;
                            m &= all >= 32 ? ~0u : all > 0 ? (1u << all) - 1 : 0u;
                            if ((dead >> (2 * c)) & 1) m &= 0xffff0000u;
                            if ((dead >> (2 * c + 1)) & 1) m &= 0x0000ffffu;
                            live[c] = m;
                        }
                    }
                    float mx = NEG;
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        float v[32];
                        tmem_ld32(ts + 32 * c, v);
                        if (edge) {
#pragma unroll
                            for (int x = 0; x < 32; x++)
                                if (!((live[c] >> x) & 1)) v[x] = NEG;
                        }
#pragma unroll
                        for (int x = 0; x < 32; x += 2) mx = fmaxf(mx, fmaxf(v[x], v[x + 1]));
                    }
                    const bool raise = mx * rs > top + kSlack;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float up = fmaxf(top, mx * rs);
                        const float c = up == top ? 1.f : ex2(top - up);
                        top = up;
                        sum *= c;
                        if (!first) {
                            const bool done = mbar_wait_spin(bar_o(st), (jobs - 1) & 1);
                            if (!__all_sync(0xffffffffu, done)) { fail(); ok = false; break; }
                            tc_fence_after();
#pragma unroll 1
                            for (int x = 0; x < D; x += 32) {
                                float v[32];
                                tmem_ld32(to + x, v);
#pragma unroll
                                for (int half = 0; half < 2; half++) {
                                    uint32_t u[16];
#pragma unroll
                                    for (int y = 0; y < 16; y++) u[y] = __float_as_uint(v[16 * half + y] * c);
                                    tmem_st16(to + x + 16 * half, u);
                                }
                            }
                            tmem_wait_st();
                        }
                    }
                    const float off = kShift - (top == NEG ? 0.f : top);
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        float v[32];
                        tmem_ld32(ts + 32 * c, v);
                        if (edge) {
#pragma unroll
                            for (int x = 0; x < 32; x++)
                                if (!((live[c] >> x) & 1)) v[x] = NEG;
                        }
                        uint32_t u[16];
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            const float a = ex2(fmaf(v[x], rs, off)), b = ex2(fmaf(v[x + 1], rs, off));
                            s0 += a; s1 += b;
                            u[x / 2] = pack2<BF>(a, b);
                        }
                        tmem_st16(ts + 16 * c, u);
                    }
                    sum += s0 + s1;
                    tmem_wait_st();
                }
                first = false;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p(st));
                jobs++;
            }
            if (!ok) break;
            // the stream's last product, then both streams' maxima and sums
            if (!first) {
                const bool done = mbar_wait_spin(bar_o(st), (jobs - 1) & 1);
                if (!__all_sync(0xffffffffu, done)) { fail(); ok = false; }
            }
            ml[(st * kTcTile + r) * 2] = top;
            ml[(st * kTcTile + r) * 2 + 1] = sum;
            if (!meet()) break;
            tc_fence_after();
            // nq = 2: this thread's row, all values; nq = 1: both streams hold the row, this thread takes a part of its values
            float w0 = 1.f, w1 = 0.f, mt = top, l = sum;
            if (w.nq == 1) {
                const float m0 = ml[r * 2], l0 = ml[r * 2 + 1], m1 = ml[(kTcTile + r) * 2], l1 = ml[(kTcTile + r) * 2 + 1];
                mt = fmaxf(m0, m1);
                w0 = m0 == mt ? 1.f : ex2(m0 - mt);
                w1 = m1 == mt ? 1.f : ex2(m1 - mt);
                l = w0 * l0 + (w.n > 1 ? w1 * l1 : 0.f);
            }
            const bool both = w.nq == 1 && w.n > 1;
            const uint32_t ta = lanes + G::O0 + (w.nq == 2 ? 128 * st : 0);
            const int x0 = w.nq == 2 ? 0 : st * (D / 2), x1 = w.nq == 2 ? D : x0 + D / 2;
            const bool marked = nan_mark[pieces & 3] == (uint32_t)pieces + 1;
            const int row = w.row0 + grow, qi = row / p.group, qh = row - qi * p.group;
            const int64_t slot = attn_slot_row<1>(blockIdx.x, w.c0, 0);
            if (warp_ok) {
#pragma unroll 1
                for (int x = x0; x < x1; x += 32) {
                    float v[32];
                    tmem_ld32(ta + x, v);
                    if (both) {
                        float v1[32];
                        tmem_ld32(lanes + G::O0 + 128 + x, v1);
#pragma unroll
                        for (int y = 0; y < 32; y++) v[y] = v[y] * w0 + v1[y] * w1;
                    }
                    if (marked) {
                        // infinities and NaN among the new tokens of this piece
                        const int a = max(w.s.ctx, w.tile0 * kTcTile), e = min(w.s.len, (w.tile0 + w.n) * kTcTile);
#pragma unroll 1
                        for (int t = a; t < e; t++) {
                            const int page = p.table[(int64_t)w.s.b * p.max_pages + (t >> p.cache.lp)];
                            if (page < 0 || page >= p.cache.n_pages) continue;
                            const int64_t crow = kv_row(p.cache, ((int64_t)page << p.cache.lp) + (t & ((1 << p.cache.lp) - 1)), w.h);
                            const bool see = (sees >> (t - w.s.ctx)) & 1;
#pragma unroll
                            for (int y = 0; y < 32; y++) {
                                const float f = tc_nonfinite<FMT, D>(p.cache, crow, x + y);
                                if (see) v[y] += f;
                            }
                        }
                    }
                    if (row_ok && w.c0 == w.c1) {
                        const float inv_l = l == 0.f ? 0.f : 1.0f / l;
                        uint16_t *dst = p.out + ((int64_t)(w.s.q0 + qi) * p.n_q + w.h * p.group + qh) * D + x;
#pragma unroll
                        for (int y = 0; y < 32; y += 8)
                            *reinterpret_cast<uint4 *>(dst + y) =
                                make_uint4(pack2<true>(v[y] * inv_l, v[y + 1] * inv_l), pack2<true>(v[y + 2] * inv_l, v[y + 3] * inv_l),
                                           pack2<true>(v[y + 4] * inv_l, v[y + 5] * inv_l), pack2<true>(v[y + 6] * inv_l, v[y + 7] * inv_l));
                    } else if (row_ok) {
                        float4 *dst = reinterpret_cast<float4 *>(p.part) + (slot * (D / 4) + x / 4) * kTcRows + grow;
#pragma unroll
                        for (int y = 0; y < 32; y += 4) dst[y / 4 * kTcRows] = make_float4(v[y], v[y + 1], v[y + 2], v[y + 3]);
                    }
                }
            }
            tc_fence_before();
            if (w.c0 != w.c1) {
                if (row_ok && (w.nq == 2 || st == 0))
                    *reinterpret_cast<float2 *>(part_ml + (slot * kTcRows + grow) * 2) = make_float2(mt, l);
                if (w.c0 == (int)blockIdx.x) set = TcSet{w.rows, w.row0, w.h, w.s.q0, w.c0, w.c1, 0, 0};
            }
            tiles_seen += w.n;
            pieces++;
        }
        if (tid == 0) reinterpret_cast<TcSet *>(p.counters)[blockIdx.x] = ok ? set : TcSet{};
    } else if (warp == kTcMmaWarp) {
        // ---------------- products ----------------
        // the whole warp walks the jobs, so that operands stay in uniform registers; one lane issues
        constexpr uint32_t TYPE = BF ? 1u : 0u;
        constexpr uint32_t IDESC = (1u << 4) | (TYPE << 7) | (TYPE << 10) | ((uint32_t)(kTcTile >> 4) << 24);
        constexpr uint32_t IDESC_S = IDESC | ((uint32_t)(kTcTile >> 3) << 17);
        constexpr uint32_t IDESC_O = IDESC | ((uint32_t)(D >> 3) << 17) | (1u << 16);     // B N-major
        const uint64_t k_desc = sw128_desc(0), v_desc = sw128_desc_mn(0, G::HALF);
        const bool one = elect_one();
        int tiles = 0, pieces = 0;
        int jobs0 = 0, jobs1 = 0;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t phase) {
            const bool r = mbar_wait_spin(bar, phase);
            if (!__all_sync(0xffffffffu, r) || *abort_flag) { fail(); ok = false; }
            return ok;
        };
        while (ok && work.next(p, w)) {
            if (!wait(bar_q, pieces & 1)) break;
            tc_fence_after();
            pieces++;
            const int nj = w.n * w.nq, two = w.nq == 2;                      // jobs: (tile, stream)
            auto scores = [&](int j) {
                const int s = j & 1, x = tc_k_pos(tiles + (two ? j >> 1 : j)), slot = x % NS;
                if ((!two || s == 0) && !wait(bar_full(slot), (x / NS) & 1)) return;
                tc_fence_after();
                const uint32_t q = (sb + G::OFF_Q + (two ? s : 0) * G::TILE) >> 4, k = (sb + G::OFF_RING + slot * G::TILE) >> 4;
                const uint32_t ds = tmem + G::S0 + 128 * s;
                if (one) {
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        const uint32_t o = ((i >> 2) * G::HALF + (i & 3) * 32) >> 4;
                        umma_f16_ss(ds, k_desc + (q + o), k_desc + (k + o), IDESC_S, i > 0);
                    }
                    umma_commit(bar_s(s));
                    if (!two || s == 1) umma_commit(bar_empty(slot));
                }
                __syncwarp();
            };
            for (int j = 0; j < 2 && j < nj && ok; j++) scores(j);
            for (int j = 0; j < nj && ok; j++) {
                const int s = j & 1, x = tc_v_pos(tiles + (two ? j >> 1 : j)), slot = x % NS;
                if (!wait(bar_p(s), (s ? jobs1 : jobs0) & 1)) break;
                if (s) jobs1++;
                else jobs0++;
                if ((!two || s == 0) && !wait(bar_full(slot), (x / NS) & 1)) break;
                tc_fence_after();
                const uint32_t v = (sb + G::OFF_RING + slot * G::TILE) >> 4;
                const uint32_t dd = tmem + G::O0 + 128 * s, pp = tmem + G::S0 + 128 * s;
                if (one) {
#pragma unroll
                    for (int i = 0; i < kTcTile / 16; i++)
                        umma_f16_ts(dd, pp + 8 * i, v_desc + (v + i * 128), IDESC_O, (j >= 2 || i > 0) ? 1u : 0u);
                    umma_commit(bar_o(s));
                    if (!two || s == 1) umma_commit(bar_empty(slot));
                }
                __syncwarp();
                if (j + 2 < nj) scores(j + 2);
            }
            tiles += w.n;
        }
        // do not free tensor memory under products still running (after an abort)
        if (jobs0 > 0) mbar_wait_spin(bar_o(0), (jobs0 - 1) & 1);
        if (jobs1 > 0) mbar_wait_spin(bar_o(1), (jobs1 - 1) & 1);
        __syncwarp();
    } else if (warp == kTcCopyWarp) {
        // ---------------- keys and values from the cache ----------------
        // a page's tokens (at most 128 of them, a box) at a time: lane i copies the tile's i-th box
        const int box = min(1 << p.cache.lp, kTcTile), boxes = kTcTile / box;
        struct Tile {
            int64_t row;            // this lane's box: its first cached row
            bool have;              // ... which exists
            unsigned valid, dead;   // boxes that exist; 16-token strips without a page
            int ctx, len, mark;     // first new token and end within the tile; mark of the piece
        };
        constexpr int RING = G::QUANT ? G::NR : NS;
        int pieces = 0, tiles = 0, lands = 0, copied = 0;                    // copied: positions up to here
        bool ok = true;
        // keys (side 0) or values (side 1) of a tile into position x
        auto copy = [&](const Tile &q, int side, int x) {
            const int slot = x % RING, turn = x / RING;
            const bool free_slot = turn == 0 || mbar_wait_spin(G::QUANT ? bar_rawe(slot) : bar_empty(slot), (turn - 1) & 1);
            if (!__all_sync(0xffffffffu, free_slot) || *abort_flag) { fail(); ok = false; return; }
            copied = x + 1;
            if constexpr (G::QUANT) {
                const uint32_t dst = sb + G::OFF_RAW + slot * G::RAW;
                if (lane == 0) {
                    // tokens present, first new one (values only), page marks, mark of the piece
                    *reinterpret_cast<int4 *>(smem + G::OFF_SIDES + 16 * slot) =
                        make_int4(q.len, side ? q.ctx : kTcTile, (int)q.dead, q.mark);
                    mbar_arrive_expect_tx(bar_rawf(slot), __popc(q.valid) * box * (G::RB + 2 * G::NB));
                }
                __syncwarp();
                if (q.have) {
                    bulk_g2s(dst + lane * box * G::RB, (side ? p.cache.v : p.cache.k) + q.row * G::RB, box * G::RB, bar_rawf(slot));
                    bulk_g2s(dst + kTcTile * G::RB + lane * box * 2 * G::NB,
                             (side ? p.cache.v_scale : p.cache.k_scale) + q.row * G::NB, box * 2 * G::NB, bar_rawf(slot));
                }
            } else {
                const uint32_t dst = sb + G::OFF_RING + slot * G::TILE;
                const bool fix = side && (q.ctx < kTcTile || q.dead);
                const uint32_t bar = fix ? bar_land : bar_full(slot);
                if (lane == 0) mbar_arrive_expect_tx(bar, __popc(q.valid) * box * G::HALVES * 128);
                __syncwarp();
                if (q.have)
#pragma unroll
                    for (int half = 0; half < G::HALVES; half++)
                        tma_box_2d(dst + half * G::HALF + lane * box * 128, side ? &vmap : &kmap, 64 * half, (int)q.row, bar);
                if (fix) {
                    // zeros behind the end and where there is no page; new tokens' infinities and NaN out, and marked
                    const bool landed = mbar_wait_spin(bar_land, lands & 1);
                    lands++;
                    if (!__all_sync(0xffffffffu, landed)) { fail(); ok = false; return; }
                    bool hit = false;
#pragma unroll 1
                    for (int i = (q.dead ? 0 : q.ctx) * (D / 8) + lane; i < kTcTile * (D / 8); i += 32) {
                        const int r = i / (D / 8), c = i % (D / 8);
                        if (r >= q.len || ((q.dead >> (r >> 4)) & 1)) {
                            sts128(dst + tc_chunk(r, c), make_uint4(0, 0, 0, 0));
                        } else if (r >= q.ctx) {
                            const uint4 v = lds128(dst + tc_chunk(r, c));
                            uint32_t u[4] = {v.x, v.y, v.z, v.w};
                            bool any = false;
#pragma unroll
                            for (int y = 0; y < 4; y++) {
                                if ((u[y] & 0x7f80u) == 0x7f80u) { u[y] &= 0xffff0000u; any = true; }
                                if ((u[y] & 0x7f800000u) == 0x7f800000u) { u[y] &= 0xffffu; any = true; }
                            }
                            if (any) { sts128(dst + tc_chunk(r, c), make_uint4(u[0], u[1], u[2], u[3])); hit = true; }
                        }
                    }
                    if (hit) nan_mark[(q.mark - 1) & 3] = (uint32_t)q.mark;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_full(slot));
                }
            }
        };
        Tile last{};
        while (ok && work.next(p, w)) {
            const int32_t *table = p.table + (int64_t)w.s.b * p.max_pages;
            auto page_of = [&](int t) {
                const int tok = t * kTcTile + lane * box;
                return (lane < boxes && tok < w.s.len) ? table[tok >> p.cache.lp] : -2;
            };
            int next_page = page_of(w.tile0);
            for (int t = w.tile0; t < w.tile0 + w.n && ok; t++) {
                const int page = next_page, tok = t * kTcTile + lane * box;
                if (t + 1 < w.tile0 + w.n) next_page = page_of(t + 1);
                Tile q;
                q.have = page >= 0 && page < p.cache.n_pages;
                q.row = q.have ? (((int64_t)page * p.cache.n_kv + w.h) << p.cache.lp) + (tok & ((1 << p.cache.lp) - 1)) : 0;
                q.valid = __ballot_sync(0xffffffffu, q.have);
                // strip i lies in box 16 i / box
                q.dead = __ballot_sync(0xffffffffu, lane < 8 && t * kTcTile + 16 * lane < w.s.len &&
                                                        !((q.valid >> (16 * (lane & 7) / box)) & 1));
                q.ctx = min(max(0, w.s.ctx - t * kTcTile), kTcTile);
                q.len = min(w.s.len - t * kTcTile, kTcTile);
                q.mark = pieces + 1;
                if (lane == 0) {
                    dead_strips[tiles & 7] = (uint8_t)q.dead;
                    if (q.dead) atomicOr(error, BQG_DEVERR_PAGE);
                }
                copy(q, 0, tc_k_pos(tiles));
                if (ok && tiles) copy(last, 1, tc_v_pos(tiles - 1));
                last = q;
                tiles++;
            }
            pieces++;
        }
        if (ok && tiles) copy(last, 1, tc_v_pos(tiles - 1));
        // do not leave while copies into shared memory are in flight (position 2 tiles - 1 is not used)
        for (int q = max(0, copied - RING); q < copied; q++)
            if (q != 2 * tiles - 1) mbar_wait_spin(G::QUANT ? bar_rawf(q % RING) : bar_full(q % RING), (q / RING) & 1);
    } else {
        // ---------------- fp16 tiles from codes and scales ----------------
        if constexpr (G::QUANT) {
            const int lt = tid - 32 * (kTcCopyWarp + 1);                     // 0 .. 255
            constexpr int STEP = 256 / G::CPT;
            const int c = lt % G::CPT, r0 = lt / G::CPT;                     // chunk c of rows r0 + i STEP
            int tiles = 0;
            bool ok = true;
            auto build = [&](int x) {
                const int rs = x % G::NR, slot = x % NS;
                bool ready = mbar_wait_spin(bar_rawf(rs), (x / G::NR) & 1);
                if (x >= NS) ready &= mbar_wait_spin(bar_empty(slot), ((x / NS) - 1) & 1);
                if (!__all_sync(0xffffffffu, ready) || *abort_flag) { fail(); ok = false; return; }
                const int4 side = *reinterpret_cast<const int4 *>(smem + G::OFF_SIDES + 16 * rs);
                const uint32_t src = sb + G::OFF_RAW + rs * G::RAW, dst = sb + G::OFF_RING + slot * G::TILE;
                bool hit = false;
#pragma unroll
                for (int i = 0; i < G::NC; i++) {
                    const int r = r0 + i * STEP;
                    const uint4 q = lds128(src + (i * 256 + lt) * 16);
                    uint32_t d;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(d) : "r"(src + kTcTile * G::RB + (r * G::NB + (FMT == BQG_Q8_0 ? c >> 1 : c)) * 2) : "memory");
                    // no token: zeros; a new token's infinite or NaN scale: zeros, and marked
                    if (r >= side.x || ((side.z >> (r >> 4)) & 1)) d = 0;
                    if (r >= side.y && (d & 0x7c00u) == 0x7c00u) { d = 0; hit = true; }
                    d |= d << 16;
                    const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
                    if constexpr (FMT == BQG_Q8_0) {
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint32_t b = wd[k] ^ 0x80808080u;
                            u[2 * k] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4140), 0x64806480u), d);
                            u[2 * k + 1] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4342), 0x64806480u), d);
                        }
                        // a row's second half of chunks stores in the other order: distinct banks
                        const uint4 lo = make_uint4(u[0], u[1], u[2], u[3]), hi = make_uint4(u[4], u[5], u[6], u[7]);
                        const int f = (c >> 2) & 1;
                        sts128(dst + tc_chunk(r, 2 * c + f), f ? hi : lo);
                        sts128(dst + tc_chunk(r, 2 * c + 1 - f), f ? lo : hi);
                    } else {
                        uint32_t u[16];                                   // value pairs of the block in order
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint32_t b = wd[k] & 0x0f0f0f0fu, e = (wd[k] >> 4) & 0x0f0f0f0fu;
                            u[2 * k] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4140), 0x64086408u), d);
                            u[2 * k + 1] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4342), 0x64086408u), d);
                            u[8 + 2 * k] = hmul2(hsub2(__byte_perm(e, 0x64646464u, 0x4140), 0x64086408u), d);
                            u[8 + 2 * k + 1] = hmul2(hsub2(__byte_perm(e, 0x64646464u, 0x4342), 0x64086408u), d);
                        }
                        const bool f = c >> 1;                            // the second 64 values: pairs of chunks swapped
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            sts128(dst + tc_chunk(r, 4 * c + (k ^ (f ? 2 : 0))),
                                   f ? make_uint4(u[4 * (k ^ 2)], u[4 * (k ^ 2) + 1], u[4 * (k ^ 2) + 2], u[4 * (k ^ 2) + 3])
                                     : make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]));
                    }
                }
                if (hit) nan_mark[(side.w - 1) & 3] = (uint32_t)side.w;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_rawe(rs));
                    mbar_arrive(bar_full(slot));
                }
            };
            while (ok && work.next(p, w))
                for (int t = 0; t < w.n && ok; t++, tiles++) {
                    build(tc_k_pos(tiles));
                    if (ok && tiles) build(tc_v_pos(tiles - 1));
                }
            if (ok && tiles) build(tc_v_pos(tiles - 1));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kTcMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Joins the pieces of the sets that several CTAs shared: 32 rows of one set
// per CTA (blockIdx.x: the set's first CTA), one row per lane, an eighth of the values
// per warp.  In the order of the CTAs.
template <int D> __global__ void __launch_bounds__(256) attn_tc_join_kernel(const AttnParams p, int ctas)
{
    pdl_wait();
    pdl_launch_dependents();
    const TcSet set = reinterpret_cast<const TcSet *>(p.counters)[blockIdx.x];
    const int row = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
    if (row >= set.rows) return;
    constexpr int V = D / 32;                                                // groups of four values per warp
    const float2 *ml = reinterpret_cast<const float2 *>(p.part + (int64_t)2 * ctas * kTcRows * D);
    const float4 *part = reinterpret_cast<const float4 *>(p.part);
    auto slot = [&](int c) { return attn_slot_row<1>(c, set.c0, 0); };
    float mt = -__builtin_huge_valf();
#pragma unroll 4
    for (int c = set.c0; c <= set.c1; c++) mt = fmaxf(mt, ml[slot(c) * kTcRows + row].x);
    float l = 0.f, v[4 * V];
#pragma unroll
    for (int i = 0; i < 4 * V; i++) v[i] = 0.f;
#pragma unroll 2
    for (int c = set.c0; c <= set.c1; c++) {
        const float2 q = ml[slot(c) * kTcRows + row];
        const float w = (q.x == mt) ? 1.f : ex2(q.x - mt);
        l += w * q.y;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float4 a = part[(slot(c) * (D / 4) + warp * V + i) * kTcRows + row];
            v[4 * i] += w * a.x; v[4 * i + 1] += w * a.y; v[4 * i + 2] += w * a.z; v[4 * i + 3] += w * a.w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int qi = (set.row0 + row) / p.group, qh = set.row0 + row - qi * p.group;
    uint16_t *dst = p.out + ((int64_t)(set.q0 + qi) * p.n_q + set.h * p.group + qh) * D + warp * 4 * V;
#pragma unroll
    for (int i = 0; i < V; i += 2)
        *reinterpret_cast<uint4 *>(dst + 4 * i) =
            make_uint4(pack2<true>(v[4 * i] * inv, v[4 * i + 1] * inv), pack2<true>(v[4 * i + 2] * inv, v[4 * i + 3] * inv),
                       pack2<true>(v[4 * i + 4] * inv, v[4 * i + 5] * inv), pack2<true>(v[4 * i + 6] * inv, v[4 * i + 7] * inv));
}

}  // namespace bqg
