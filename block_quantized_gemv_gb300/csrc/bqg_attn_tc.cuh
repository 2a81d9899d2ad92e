// bqg_attn_tc.cuh -- the same attention for many rows per KV head, on tcgen05.
//
// With R = new tokens x heads of a group rows sharing a KV head, the two
// products cost R multiply-adds per cached value: from a few dozen rows on the
// tensor cores and not the stream decide, and mma.sync cannot feed them.
// Here a tile is 128 cached tokens against 128 rows (the MMA's M):
//     S = Q K^T  (N = tokens, K = D),   O += P V  (N = D, K = tokens)
// with Q, K and V in shared memory (128-byte swizzle; V is the N-major operand
// as it lies, tokens x values), and S, P and O in tensor memory: P takes
// the place of S, two fp16 or bf16 per column, and is the second product's A operand.
//
//  * Two streams share a CTA, each with its own rows of O, maximum and sum.  With more than
//    128 rows in a row group (bf16: up to 256) they are its two halves over the
//    same keys and values, and a tile is taken as two steps of 64 tokens; with at most 128 they
//    are the two halves of each tile's tokens, joined at the end, and a tile is one step.
//    Tensor memory holds two buffers of 2 x 64 scores per row, so the products of the next step
//    run under the softmax of this one (one buffer of 128 tokens per stream
//    left both waiting for each other's latency: 4240 cycles per 128 tokens
//    x 256 rows, 2048 of them products).
//  * head_dim 256 leaves room for one stream of 128 rows (256 columns of O, two buffers of 64 scores), so a tile is 64 tokens
//    and one step, and warps 4-7 have nothing to do.
//  * Warps 0-3 and 4-7: softmax of stream 0 and 1, one row per thread, its 64 scores
//    in registers.  The running maximum is raised only when exceeded by kSlack
//    (see bqg_attn.cuh), and only then is O rescaled, after the products so far.
//  * Warp 8 issues the products: for each step its values and the
//    scores of the step after next, behind one wait for all they need and with
//    one commit.  (A wait that is already over costs this warp 100 to 200 cycles and a commit 30 to
//    120, so a step per stream with three waits took 1230 cycles for 640 of products.)
//  * Warp 10 plans the CTA's pieces; warp 9 brings keys, warp 11 values.  bf16: straight into the ring of tiles, in TMA boxes
//    of 64 values x the tokens of a page.  q8_0 / q4_0: codes and scales as they
//    lie, one bulk copy each per page, into a ring of their own, from which warps
//    12-19 build the tile: codes as fp16 integers (bqg_attn.cuh), times the
//    block's scale: one rounding (relative 2^-11, for keys too: a block's scale
//    cannot be applied behind a product that sums over all blocks).
//  * Tiles are shared out over the CTAs, a tile of two halves counting twice: one piece for each, or even
//    ranges (see TcWork).  Sets of tiles that several CTAs share leave partial
//    results, which a second, small launch joins: with up to 256 rows of
//    them, the CTA that came last took longer for it than the whole GPU does.
//  * Every wait is bounded; one that gives up sets the error word, and the
//    rest of the CTA's work is skipped.
//  * Measured (head_dim 128, back to back): bf16, 4 x 16,384 tokens, 64 new, 8 heads on each of 8: 128 us, 1080 TFLOP/s; a step of
//    64 tokens x 256 rows takes 2000 cycles, 1400 of them products (N = 64: each MMA reads its 128 x 16 of Q, 56 cycles
//    instead of 32).  q8_0, 8 x 5000, 13 new, 4 heads on each of 8: 34.5 us: 7 until the first scores, 1.4 per tile of
//    128 tokens (building its two sides, 1100 to 1300 cycles each), 2 for the results, 3 for the join.  Two
//    teams of builders, one per side, took 34 % longer.  head_dim 256, 8 x 4000, 64 new: bf16 84 us, q8_0 98 (mma.sync in
//    16 turns of 16 rows: 270, 276).
//
// A drafted token's infinite or NaN value, or one beyond fp16's range, must not reach rows that do not see
// it, and 0 x NaN or 0 x inf in the product would.  In tiles that hold new tokens zeros
// are stored for such values and the piece is marked; the rows that see the
// token add them (infinities and NaN stay what they are, what fp16 cannot hold is an infinity) when they are written.
#pragma once

#include <cuda.h>

#include "bqg_attn.cuh"
#include "bqg_tc.cuh"

namespace bqg {

constexpr int kTcHalf = 128;             // rows of a stream
constexpr int kTcMmaWarp = 8, kTcKeyWarp = 9, kTcPlanWarp = 10, kTcValueWarp = 11, kTcBuildWarp = 12;
constexpr int kTcAhead = 2;              // tiles whose scores may be issued before the first values are needed
constexpr int kTcMarks = 32;             // tiles or pieces that the copying warps may be ahead of the softmax

// A set of tiles shared by several CTAs, as its first CTA describes it for the join (rows 0: none).
struct TcSet {
    int rows, row0, h, q0;      // rows of the group, the first one; KV head; the sequence's first query token
    int c0, c1;                 // CTAs
    int lo, pad;                // tokens left out (SharedSeq)
};

template <int FMT, int D> struct TcGeom {
    static constexpr bool QUANT = FMT != BQG_BF16;
    // head_dim 256: one stream, since two would not fit in tensor memory, and tiles of 64 tokens, a step each
    static constexpr bool SINGLE = D == 256;
    static constexpr int TT = SINGLE ? 64 : 128;                        // tokens of a tile
    static constexpr int STREAMS = SINGLE ? 1 : 2;
    static constexpr int SOFT = 4 * STREAMS;                            // softmax warps
    static constexpr int BUILD_WARPS = QUANT ? 8 : 0;
    static constexpr int THREADS = 32 * (kTcBuildWarp + BUILD_WARPS);
    // registers per thread at launch, and what the warpgroups make of them: 640 threads x 96 =
    // 256 x 144 (softmax) + 128 x 64 (products, copies) + 256 x 64 (building)
    static constexpr int REGS_SOFTMAX = 144, REGS_OTHER = 64;
    static_assert(!QUANT || 256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * 96, "register split");
    // halves of a row group: quantized tiles leave room for one tile of queries
    static constexpr int NQ = QUANT || SINGLE ? 1 : 2;
    static constexpr int ROWS = NQ * kTcHalf;                           // rows of a row group
    static constexpr int HALVES = D / 64;                               // 64 values: one 128-byte swizzle atom wide
    static constexpr int QHALF = kTcHalf * 128, HALF = TT * 128;        // bytes of 64 values of a tile of Q, of K or V
    static constexpr int QTILE = HALVES * QHALF, TILE = HALVES * HALF;
    static constexpr int NS = (D == 64) ? 6 : (SINGLE && FMT == BQG_Q8_0) ? 3 : 4;   // ring slots (see tc_k_pos)
    static constexpr int RB = KvRow<FMT, D>::BYTES;
    static constexpr int NB = D / QK;
    static constexpr int CPT = RB / 16;                                 // 16-byte chunks of a cached row
    static constexpr int CHUNKS = TT * CPT;                        // of a side (a tile's keys or values)
    static constexpr int RAW = QUANT ? TT * (RB + 2 * NB) : 0;     // codes, then scales, of a side
    static constexpr int NR = !QUANT ? 0 : (SINGLE || RAW > 16384) ? 3 : 5;         // raw sides in flight: 23 to 51 KiB
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = NQ * QTILE;
    static constexpr int OFF_RAW = OFF_RING + NS * TILE;
    static constexpr int OFF_ML = OFF_RAW + NR * RAW;                   // (maximum, sum) per stream and row
    static constexpr int OFF_SIDES = OFF_ML + 2 * kTcHalf * 8;          // what a raw side holds, 16 bytes each
    static constexpr int OFF_RS = OFF_SIDES + 16 * NR;                  // softmax scale per row
    static constexpr int OFF_PIECES = OFF_RS + (QUANT ? kTcHalf * 4 : 0);   // two pieces
    static constexpr int OFF_BARS = OFF_PIECES + 2 * 64;
    // full, empty per slot; raw full, empty; products done, probabilities (two each);
    // queries; the softmax warps' meeting point; values landed; piece there, taken (two each)
    static constexpr int NBARS = 2 * NS + 2 * NR + 4 + 3 + 4;
    static constexpr int OFF_WORDS = OFF_BARS + NBARS * 8;              // tensor memory base, NaN marks, page marks
    static constexpr int SMEM = OFF_WORDS + 8 + 4 * kTcMarks + kTcMarks + 1024;   // + slack for 1024-byte alignment
    static constexpr int S0 = 0, O0 = 256;                              // tensor memory columns, + 128 per stream
    static_assert(SMEM <= 232448, "shared memory");
};

// Ring positions of the keys and values of tile t of a piece of n tiles, in the order in which the products
// take them: K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1); `before`: tiles of the CTA's earlier pieces.  Position x lies
// in slot x % slots, in the slot's phase x / slots.  A phase's parity tells nothing to who may be two
// phases off, so whoever waits for a slot's phase has to know that the one before is complete.
//  * Quantized: a CTA's positions are numbered through.  The build warps take them in this order, so who has seen position
//    x - 3 of the raw ring emptied knows it of all before; consecutive positions of keys (or
//    values) are at most 3 apart, no more than the ring has slots.  (With the numbers of bf16 a key warp
//    that saw a piece's last values emptied knew nothing of the next one's first keys.)
//  * bf16: a slot serves keys or values only (but for the very first keys), so each copying warp has
//    waited for every phase of its slots; numbered through all pieces, the last values before the next piece's
//    first keys leave the position before theirs to them.
template <bool QUANT> __device__ __forceinline__ int tc_k_pos(int before, int t)
{
    if constexpr (QUANT) return 2 * before + (t < kTcAhead ? t : 2 * t - 1);
    return before + t < kTcAhead ? before + t : 2 * (before + t) - 1;
}
template <bool QUANT> __device__ __forceinline__ int tc_v_pos(int before, int t, int n)
{
    if constexpr (QUANT) return 2 * before + (t == n - 1 ? 2 * n - 1 : 2 * t + 2);
    return 2 * (before + t) + 2;
}

// The pieces of one CTA: consecutive tiles of one (sequence, KV head, row group).
template <typename Seq> struct alignas(16) TcPieceOf {
    Seq s;
    int h, row0, rows;          // first row of the group, its rows
    int nq;                     // 2: the streams are two halves of the rows; 1: of each tile's tokens
    int tile0, n;               // tiles of the piece
    int c0, c1;                 // CTAs that share the (sequence, KV head, row group)
};
// Units: tiles x streams.  Where it costs at most kTcSecond units more than an even share, no CTA
// takes more than one piece: a second one waits for its queries, its first keys and an
// idle tensor core, 8 to 9 us, the time of 5 quantized units or 10 of bf16.  Otherwise (more (sequence, KV head, row group)
// than CTAs, or few of unlike lengths) each takes an equal range of the line of all units.
// 8 x 5000 tokens q8_0, 64 such groups on 152 CTAs: 46 us with one piece each, 50 with ranges.
template <int NQ> constexpr int kTcSecond = NQ == 2 ? 10 : 5;
static_assert(sizeof(TcPieceOf<AttnSeq>) == 64 && sizeof(TcPieceOf<SharedSeq>) == 64, "two pieces in shared memory");
template <int NQ, int TT, typename P> struct TcWork {
    using Seq = typename P::Seq;
    using TcPiece = TcPieceOf<Seq>;
    int64_t per, cur, end, base;
    int most;                   // units of a piece where each CTA has one; 0: ranges of `per` units
    Seq s;
    // tiles of a sequence
    __device__ static __forceinline__ unsigned tiles_of(const Seq &q) { return (q.len + TT - 1) / TT - attn_lo(q) / TT; }
    __device__ static __forceinline__ int64_t cost(const P &p, const Seq &q)
    {
        const int tiles = tiles_of(q), halves = (q.T * p.group + kTcHalf - 1) / kTcHalf;
        return (int64_t)p.cache.n_kv * tiles * halves;
    }
    // pieces of at most `most` units (a multiple of NQ) of a KV head: of a row group with NQ halves, of one with fewer, of all
    struct Pieces { int groups, full, rest, head; };
    __device__ static __forceinline__ Pieces pieces(const P &p, const Seq &q, int most)
    {
        const unsigned tiles = tiles_of(q), halves = (q.T * p.group + kTcHalf - 1) / kTcHalf;
        Pieces r;
        r.groups = halves / NQ;
        r.full = (tiles * NQ + most - 1) / (unsigned)most;
        r.rest = halves % NQ ? (tiles + most - 1) / (unsigned)most : 0;
        r.head = r.groups * r.full + r.rest;
        return r;
    }
    __device__ __forceinline__ void init(const P &p, int lane, int &bad)
    {
        auto weight = [&](const Seq &q) { return cost(p, q); };
        int64_t mine, total;
        // One set of tokens (a prefix of all sequences, one sequence) needs no look at others: sums and searches over lanes are most of
        // the planning's instructions.
        const bool one = (P::SHARED || NQ == 2) && p.n_seq == 1;
        if (one) {
            s = attn_seq(p, 0, bad);
            total = cost(p, s);
        } else {
            total = attn_total(p, lane, weight, bad, s, mine);
        }
        // at least NQ, so that every range between a set's first and last holds the beginning of a tile
        per = max(div_pos(total + gridDim.x - 1, gridDim.x), (int64_t)NQ);
        most = 0;
        auto count = [&](int m) {
            int ignored = 0;
            if (one) return (unsigned)(p.cache.n_kv * pieces(p, s, m).head);
            unsigned n = lane < p.n_seq ? p.cache.n_kv * pieces(p, s, m).head : 0;
            for (int b = lane + 32; b < p.n_seq; b += 32) n += p.cache.n_kv * pieces(p, attn_seq(p, b, ignored), m).head;
            return __reduce_add_sync(0xffffffffu, n);
        };
        unsigned pieces_all = 0;
        if (total < (1 << 28) && (int64_t)p.n_seq * p.cache.n_kv <= gridDim.x) {
            // The smallest that leaves no CTA a second piece.  A few are tried one after the other, by one copy of the code: this runs once and
            // mostly waits for its instructions.  (Not in the quantized kernels of bqg_tree_attention: their registers are at
            // the limit, and with this they took up to 5 % longer.)
            const int first = ((int)per + NQ - 1) / NQ, last = ((int)per + kTcSecond<NQ>) / NQ;
            if constexpr (P::SHARED || NQ == 2) {
#pragma unroll 1
                for (int m = first; m <= last && !most; m++) {
                    pieces_all = count(m * NQ);
                    if (pieces_all <= gridDim.x) most = m * NQ;
                }
            } else if (count(last * NQ) <= gridDim.x) {
                int lo = first - 1, hi = last;
                while (hi - lo > 1) {
                    const int m = (lo + hi) >> 1;
                    (count(m * NQ) <= gridDim.x ? hi : lo) = m;
                }
                most = hi * NQ;
            }
        }
        if (most) {
            auto number = [&](const Seq &q) { return (int64_t)p.cache.n_kv * pieces(p, q, most).head; };
            cur = blockIdx.x;
            end = min(cur + 1, (int64_t)(P::SHARED || NQ == 2 ? pieces_all : count(most)));
            base = 0;
            if (one) return;
            mine = lane < p.n_seq ? number(s) : 0;
            if (cur < end) s = attn_find(p, cur, lane, number, s, mine, base);
            return;
        }
        cur = per * blockIdx.x;
        end = min(cur + per, total);
        base = 0;
        if (!one && cur < end) s = attn_find(p, cur, lane, weight, s, mine, base);
    }
    __device__ __forceinline__ bool next(const P &p, TcPiece &o)
    {
        if (most) {
            if (cur >= end) return false;
            const Pieces n = pieces(p, s, most);
            const unsigned off = (unsigned)(cur - base), rem = off % (unsigned)n.head;
            const unsigned tiles = tiles_of(s);
            o.h = off / (unsigned)n.head;
            const int g = min((int)(rem / (unsigned)n.full), n.groups);
            const unsigned j = rem - g * n.full, k = g < n.groups ? n.full : n.rest;               // piece j of k
            o.row0 = g * NQ * kTcHalf;
            o.rows = min(NQ * kTcHalf, s.T * p.group - o.row0);
            o.nq = g < n.groups ? NQ : 1;
            o.tile0 = j * (tiles / k) + min(j, tiles % k);
            o.n = tiles / k + (j < tiles % k);
            o.c0 = blockIdx.x - j;
            o.c1 = o.c0 + k - 1;
            o.tile0 += attn_lo(s) / TT;
            o.s = s;
            cur = end;
            return true;
        }
        int ignored = 0;
        while (cur < end) {
            while (cur - base >= cost(p, s)) {
                base += cost(p, s);
                s = attn_seq(p, s.b + 1, ignored);
            }
            const int tiles = tiles_of(s), all = s.T * p.group;
            const int halves = (all + kTcHalf - 1) / kTcHalf, groups = (halves + NQ - 1) / NQ;
            const int64_t off = cur - base, head = (int64_t)tiles * halves;
            o.h = (int)div_pos(off, head);
            const int64_t rem = off - o.h * head;
            const int g = min((int)div_pos(rem, NQ * (int64_t)tiles), groups - 1);
            o.row0 = g * NQ * kTcHalf;
            o.rows = min(NQ * kTcHalf, all - o.row0);
            o.nq = o.rows > kTcHalf ? 2 : 1;
            const int64_t seg = base + o.h * head + (int64_t)g * NQ * tiles;      // its first tile's number
            o.tile0 = (int)((cur - seg + o.nq - 1) >> (o.nq - 1));                // tiles that begin in this range
            const int last = (int)min((int64_t)tiles, (end - seg + o.nq - 1) >> (o.nq - 1));
            o.n = last - o.tile0;
            cur = seg + (int64_t)max(last, o.tile0) * o.nq;
            if (o.n <= 0) continue;
            o.c0 = (int)div_pos(seg, per);
            o.c1 = (int)div_pos(seg + (int64_t)(tiles - 1) * o.nq, per);
            o.tile0 += attn_lo(s) / TT;
            o.s = s;
            return true;
        }
        return false;
    }
};

// N-major operand (V: tokens x values, 128-byte swizzle): 64 values x 8
// tokens per atom; the next 64 values are `half` bytes on, the next 8 tokens 1024.
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
// 32 lanes x 32 columns of tensor memory (this warp's lane quarter) into registers; complete after tmem_wait_ld on them
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
// (the registers pass through, so that nothing that uses them can be placed before the wait)
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
                   "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
                   "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
template <int N> __device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void tma_box_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Byte offset of 16-byte chunk c (eight values) of row r in a swizzled tile of ROWS rows.
template <int ROWS> __device__ __forceinline__ uint32_t tc_chunk(int r, int c)
{
    return (uint32_t)((c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Zeros for the infinities and NaN among fp16 values that this thread stored: chunks c0 .. c0 + N - 1 of rows r0, r0 + step, ...
// (M of them) from row `from` on.  Not inlined: in the builders' code it took 2 to 4 % where every tile holds new tokens, though
// no value was beyond fp16 (64 x 300 tokens, 8 new, head_dim 64, q8_0: 42.8 us instead of 41.2).
template <int TT, int M, int N> __device__ __noinline__ void tc_drop_nonfinite(uint32_t dst, int r0, int step, int from, int c0)
{
#pragma unroll 1
    for (int i = 0; i < M; i++) {
        if (r0 + i * step < from) continue;
#pragma unroll 1
        for (int k = 0; k < N; k++) {
            const uint32_t chunk = dst + tc_chunk<TT>(r0 + i * step, c0 + k);
            const uint4 v = lds128(chunk);
            uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; y++) {
                if ((u[y] & 0x7c00u) == 0x7c00u) u[y] &= 0xffff0000u;
                if ((u[y] & 0x7c000000u) == 0x7c000000u) u[y] &= 0xffffu;
            }
            sts128(chunk, make_uint4(u[0], u[1], u[2], u[3]));
        }
    }
}

// Value `dim` of cached row `row`, as far as it is an infinity or NaN in the products' type; 0 otherwise.
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
    if constexpr (FMT == BQG_BF16) return isfinite(f) ? 0.f : f;
    else return fabsf(f) < 65520.f ? 0.f : f * __int_as_float(0x7f800000);    // 65520 and above round to an infinity in fp16
}

// Whether this launch's rows are the call's results.
__device__ __forceinline__ bool tc_own(const AttnParams &) { return true; }
__device__ __forceinline__ bool tc_own(const SharedParams &p) { return p.own; }

// Partial results of a piece: values in groups of four, [slot][D / 4][rows][4] (a warp's 32 rows are then
// 512 contiguous bytes), and (maximum, sum) [slot][rows].
template <int FMT, int D, typename P = AttnParams>
__global__ void __launch_bounds__(TcGeom<FMT, D>::THREADS, 1)
attn_tc_kernel(const P p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int *error)
{
    using G = TcGeom<FMT, D>;
    using TcPiece = TcPieceOf<typename P::Seq>;
    constexpr bool BF = (FMT == BQG_BF16);
    constexpr float NEG = -__builtin_huge_valf();
    constexpr float kShift = BF ? 0.0f : 8.0f;
    constexpr int NS = G::NS, NR = G::NR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bars = sb + G::OFF_BARS;
    auto bar_full = [&](int i) { return bars + 8 * i; };
    auto bar_empty = [&](int i) { return bars + 8 * (NS + i); };
    auto bar_rawf = [&](int i) { return bars + 8 * (2 * NS + i); };
    auto bar_rawe = [&](int i) { return bars + 8 * (2 * NS + NR + i); };
    const uint32_t bars2 = bars + 8 * (2 * NS + 2 * NR);
    // Commit number c of the products: the scores of step m of a piece are number C + m (C: at the piece's
    // beginning), its values number C + m + 2, which also covers the scores of step m + 2.  Number c
    // completes bar_s(c & 1) for the (c >> 1)-th time; who waits for c has waited for c - 2.
    auto bar_s = [&](int c) { return bars2 + 8 * (c & 1); };
    auto bar_p = [&](int n) { return bars2 + 16 + 8 * (n & 1); };
    const uint32_t bar_q = bars2 + 32, bar_meet = bars2 + 40, bar_land = bars2 + 48;
    auto bar_pf = [&](int n) { return bars2 + 56 + 8 * (n & 1); };
    auto bar_pe = [&](int n) { return bars2 + 72 + 8 * (n & 1); };
    volatile uint32_t *const base_word = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_WORDS);
    volatile uint32_t *const nan_mark = base_word + 2;                                                   // [piece % kTcMarks]
    volatile uint8_t *const dead_strips = reinterpret_cast<volatile uint8_t *>(base_word + 2 + kTcMarks); // [tile % kTcMarks]

    volatile float *const row_scale = reinterpret_cast<volatile float *>(smem + G::OFF_RS);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(bar_full(i), G::QUANT ? G::BUILD_WARPS : 1);
            mbar_init(bar_empty(i), 1);                // tcgen05.commit
        }
        for (int i = 0; i < NR; i++) {
            mbar_init(bar_rawf(i), 1);
            mbar_init(bar_rawe(i), G::BUILD_WARPS);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar_s(i), 1);                    // tcgen05.commit
            mbar_init(bar_p(i), G::SOFT);
            mbar_init(bar_pf(i), 1);
            mbar_init(bar_pe(i), G::SOFT + 3 + G::BUILD_WARPS);
        }
        mbar_init(bar_q, G::SOFT);
        mbar_init(bar_meet, G::SOFT);
        mbar_init(bar_land, 1);
        for (int i = 0; i < kTcMarks; i++) nan_mark[i] = 0;
        mbar_fence_init();
    }
    if (warp == kTcMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + G::OFF_WORDS), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *base_word;
    pdl_wait();                              // (own_kernel relies on this order)
    pdl_launch_dependents();

    // a wait that gives up ends its role's work; every other wait then gives up in its turn
    auto wait = [&](uint32_t bar, uint32_t phase) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_spin(bar, phase));
        if (!ok && lane == 0) atomicOr(error, 2);
        return ok;
    };
    // the next piece from the planning warp into w (whose fields that a role does not use cost it nothing); false: the last was
    TcPiece w;
    int taken = 0;
    bool ok = true;
    auto next = [&]() {
        if (!(ok = wait(bar_pf(taken), (taken >> 1) & 1))) return false;
        w = *reinterpret_cast<const TcPiece *>(smem + G::OFF_PIECES + (taken & 1) * sizeof(TcPiece));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_pe(taken));
        taken++;
        return w.n > 0;
    };

    if (warp < G::SOFT) {
        // ---------------- softmax and results ----------------
        if constexpr (G::QUANT) regs_more<G::REGS_SOFTMAX>();
        const int st = warp >> 2, r = (warp & 3) * 32 + lane;                // stream, row of its half
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = lanes + G::O0 + 128 * st;
        float *const ml = reinterpret_cast<float *>(smem + G::OFF_ML);
        float *const part_ml = p.part + (int64_t)2 * gridDim.x * G::ROWS * D;
        TcSet set{};                                                         // begun here, ended elsewhere
        int pieces = 0, tiles = 0, commits = 0, steps = 0;                   // before this piece
        // of the piece being worked on
        int grow = 0, row = 0, qi = 0, qh = 0;
        bool row_ok = false, warp_ok = false;
        unsigned long long sees = 0;
        float top = NEG, sum = 0.f;
        auto results = [&](const TcPiece &d) {
            if (!(ok = wait(bar_meet, pieces & 1))) return;
            tc_fence_after();
            // nq = 2: this thread's row, all values; nq = 1: both streams hold the row, this thread takes half of its values
            float w0 = 1.f, w1 = 0.f, mt = top, l = sum;
            const bool both = !G::SINGLE && d.nq == 1;
            if (both) {
                const float m0 = ml[r * 2], l0 = ml[r * 2 + 1], m1 = ml[(kTcHalf + r) * 2], l1 = ml[(kTcHalf + r) * 2 + 1];
                mt = fmaxf(m0, m1);
                w0 = m0 == mt ? 1.f : ex2(m0 - mt);
                w1 = m1 == mt ? 1.f : ex2(m1 - mt);
                l = w0 * l0 + w1 * l1;
            }
            const uint32_t ta = lanes + G::O0 + (both ? 0 : 128 * st);
            const int x0 = both ? st * (D / 2) : 0, x1 = both ? x0 + D / 2 : D;
            const bool marked = nan_mark[pieces % kTcMarks] == (uint32_t)pieces + 1;
            const int64_t slot = attn_slot_row<1>(blockIdx.x, d.c0, 0);
            float lj = l;                                                    // with the shared tokens'
            if (warp_ok) {
#pragma unroll 1
                for (int x = x0; x < x1; x += 32) {
                    uint32_t u[32];
                    float v[32];
                    tmem_ld32_nowait(ta + x, u);
                    if (both) {
                        uint32_t u1[32];
                        tmem_ld32_nowait(lanes + G::O0 + 128 + x, u1);
                        tmem_wait_ld(u);
                        tmem_wait_ld(u1);
#pragma unroll
                        for (int y = 0; y < 32; y++) v[y] = __uint_as_float(u[y]) * w0 + __uint_as_float(u1[y]) * w1;
                    } else {
                        tmem_wait_ld(u);
#pragma unroll
                        for (int y = 0; y < 32; y++) v[y] = __uint_as_float(u[y]);
                    }
                    if (marked) {
                        // infinities and NaN among the new tokens of this piece
                        const int a = max(d.s.ctx, d.tile0 * G::TT), e = min(d.s.len, (d.tile0 + d.n) * G::TT);
#pragma unroll 1
                        for (int t = a; t < e; t++) {
                            const int page = p.table[(int64_t)attn_table_row(d.s) * p.max_pages + (t >> p.cache.lp)];
                            if (page < 0 || page >= p.cache.n_pages) continue;
                            const int64_t crow = kv_row(p.cache, ((int64_t)page << p.cache.lp) + (t & ((1 << p.cache.lp) - 1)), d.h);
                            const bool see = (sees >> (t - d.s.ctx)) & 1;
#pragma unroll
                            for (int y = 0; y < 32; y++) {
                                const float f = tc_nonfinite<FMT, D>(p.cache, crow, x + y);
                                if (see) v[y] += f;
                            }
                        }
                    }
                    if constexpr (P::SHARED)
                        if (row_ok && d.c0 == d.c1) {
                            const int64_t at = shared_row(p, d.s, d.h, row);
                            float4 *shared = shared_at<D>(p, at, x / 4);
                            if (!p.own) {
#pragma unroll
                                for (int y = 0; y < 32; y += 4) shared[y / 4 * 32] = make_float4(v[y], v[y + 1], v[y + 2], v[y + 3]);
                            } else if (d.s.lo) {
                                const float2 q = *reinterpret_cast<const float2 *>(p.rows_ml + at * 2);
                                const float up = fmaxf(mt, q.x);
                                const float a = mt == up ? 1.f : ex2(mt - up), b = q.x == up ? 1.f : ex2(q.x - up);
                                if (x == x0) lj = l * a + q.y * b;
#pragma unroll
                                for (int y = 0; y < 32; y += 4) {
                                    const float4 f = shared[y / 4 * 32];
                                    v[y] = v[y] * a + f.x * b; v[y + 1] = v[y + 1] * a + f.y * b;
                                    v[y + 2] = v[y + 2] * a + f.z * b; v[y + 3] = v[y + 3] * a + f.w * b;
                                }
                            }
                        }
                    if (P::SHARED && !tc_own(p) && d.c0 == d.c1) {
                        // (a prefix's rows have been written)
                    } else if (row_ok && d.c0 == d.c1) {
                        const float l = lj;
                        const float inv_l = l == 0.f ? 0.f : 1.0f / l;
                        uint16_t *dst = p.out + ((int64_t)(d.s.q0 + qi) * p.n_q + d.h * p.group + qh) * D + x;
#pragma unroll
                        for (int y = 0; y < 32; y += 8)
                            *reinterpret_cast<uint4 *>(dst + y) =
                                make_uint4(pack2<true>(v[y] * inv_l, v[y + 1] * inv_l), pack2<true>(v[y + 2] * inv_l, v[y + 3] * inv_l),
                                           pack2<true>(v[y + 4] * inv_l, v[y + 5] * inv_l), pack2<true>(v[y + 6] * inv_l, v[y + 7] * inv_l));
                    } else if (row_ok) {
                        float4 *dst = reinterpret_cast<float4 *>(p.part) + (slot * (D / 4) + x / 4) * G::ROWS + grow;
#pragma unroll
                        for (int y = 0; y < 32; y += 4) dst[y / 4 * G::ROWS] = make_float4(v[y], v[y + 1], v[y + 2], v[y + 3]);
                    }
                }
            }
            tc_fence_before();
            if constexpr (P::SHARED)
                if (!p.own && d.c0 == d.c1 && row_ok && (d.nq == 2 || st == 0))
                    *reinterpret_cast<float2 *>(p.rows_ml + shared_row(p, d.s, d.h, row) * 2) = make_float2(mt, l);
            if (d.c0 != d.c1) {
                if (row_ok && (d.nq == 2 || st == 0))
                    *reinterpret_cast<float2 *>(part_ml + (slot * G::ROWS + grow) * 2) = make_float2(mt, l);
                if (d.c0 == (int)blockIdx.x) set = TcSet{d.rows, d.row0, d.h, d.s.q0, d.c0, d.c1, attn_lo(d.s), 0};
            }
            tiles += d.n;
            pieces++;
        };
        // Queries into shared memory, a row per CPR lanes: chunks per row, rows per step; bf16: the warp's 32 rows as they are; else
        // rows that serve both streams, if there are two.
        constexpr int CPR = D / 8, RPI = 32 / CPR;
        constexpr int QROWS = BF ? 32 : kTcHalf / G::SOFT, N = QROWS * CPR / 32;
        auto query_of = [&](int first) {                                     // this lane's row's, or -1
            const int qrow = w.row0 + (BF ? (w.nq == 2 ? st * kTcHalf : 0) + r : first + lane % QROWS), i0 = qrow / p.group;
            return qrow < w.row0 + w.rows
                       ? (int64_t)(w.s.q0 + i0) * p.q_stride + (int64_t)(w.h * p.group + qrow - i0 * p.group) * D : -1;
        };
        // bf16: a piece's queries are asked for before the results of the one before (d) are written, whose products are complete by
        // then (64 x 300 tokens, 16 new: 40.6 us, 45.0 otherwise; quantized, where they still have to be converted, 0 to 5 % slower).
        TcPiece before;
        bool have = false;
        for (;;) {
            if constexpr (BF) {
                const bool more = next();
                if (!ok) break;
                if (more) {
                    const int first = (warp & 3) * 32, c = lane % CPR;
                    const int64_t mine = query_of(first);
                    const uint32_t dst = sb + G::OFF_Q + (w.nq == 2 ? st : 0) * G::QTILE;
#pragma unroll 4
                    for (int n = 0; n < N; n++) {
                        const int64_t from = __shfl_sync(0xffffffffu, mine, n * RPI + lane / CPR);
                        if (st == 0 || w.nq == 2)
                            cp_async16(dst + tc_chunk<kTcHalf>(first + n * RPI + lane / CPR, c), p.q + (from >= 0 ? from + 8 * c : 0), from >= 0 ? 16 : 0);
                    }
                    cp_async_commit();
                }
                if (have) results(before);
                if (!ok || !more) break;
                before = w;
                have = true;
            } else {
                if (!next()) break;
            }
            const TcPiece &d = BF ? before : w;
            grow = d.nq == 2 ? st * kTcHalf + r : r;                         // row of the group
            row_ok = grow < d.rows;
            warp_ok = __any_sync(0xffffffffu, row_ok);
            row = d.row0 + grow;
            qi = row / p.group;
            qh = row - qi * p.group;
            sees = row_ok ? attn_sees(p, d.s, row) : 0;
            if constexpr (BF) {
                cp_async_wait<0>();
            } else {
                const int first = warp * QROWS, c = lane % CPR;
                const int64_t mine = query_of(first);
                const uint32_t dst = sb + G::OFF_Q;
                constexpr int B = N < 16 ? N : 16;
#pragma unroll 1
                for (int n = 0; n < N; n += B) {
                    uint4 v[B];
#pragma unroll
                    for (int i = 0; i < B; i++) {
                        const int64_t from = __shfl_sync(0xffffffffu, mine, (n + i) * RPI + lane / CPR);
                        v[i] = from >= 0 ? *reinterpret_cast<const uint4 *>(p.q + from + 8 * c) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < B; i++) sts128(dst + tc_chunk<kTcHalf>(first + (n + i) * RPI + lane / CPR, c), v[i]);
                }
                // two lanes per row: its largest value, the power of two, fp16
                __syncwarp();
#pragma unroll 1
                for (int r2 = first + (lane >> 1); r2 < first + QROWS; r2 += 16) {
                    auto at = [&](int k) { return dst + tc_chunk<kTcHalf>(r2, (lane & 1) * 4 + (k & 3) + (k >> 2) * 8); };
                    uint32_t hi = 0;                                     // bf16 without sign order as integers
#pragma unroll
                    for (int k = 0; k < CPR / 2; k++) {
                        const uint4 x = lds128(at(k));
                        hi = __vmaxu2(hi, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
                    }
                    hi = max(hi >> 16, hi & 0xffffu);
                    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
                    float inv = 1.f, scale = p.scale_log2;
                    if (hi > 0 && hi < 0x7f80u) {
                        const uint32_t ex = min(hi >> 7, 253u);
                        inv = __uint_as_float((254u - ex) << 23);
                        scale = fmaxf(p.scale_log2 * (1.0f / inv), 1.17549435e-38f);
                    }
                    if ((lane & 1) == 0) row_scale[r2] = scale;
#pragma unroll 2
                    for (int k = 0; k < CPR / 2; k++) {
                        float f[8];
                        bf16x8_to_f32(lds128(at(k)), f);
                        sts128(at(k), make_uint4(pack2<false>(f[0] * inv, f[1] * inv), pack2<false>(f[2] * inv, f[3] * inv),
                                                 pack2<false>(f[4] * inv, f[5] * inv), pack2<false>(f[6] * inv, f[7] * inv)));
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_q);

            const int np = d.n * d.nq;                                       // steps
            top = NEG;
            sum = 0.f;
            float rs = p.scale_log2;                                         // softmax scale of the row
            for (int m = 0; m < np; m++) {
                const int c = commits + m, i = d.nq == 2 ? m >> 1 : m, half = d.nq == 2 ? m & 1 : st;   // of the tile's tokens
                if (!(ok = wait(bar_s(c), (c >> 1) & 1))) break;
                tc_fence_after();
                // (the products that were waited for were issued after all warps had brought their queries)
                if (!BF && m == 0) rs = row_scale[r];
                const uint32_t ts = lanes + G::S0 + 128 * (c & 1) + 64 * st;
                const int tok0 = (d.tile0 + i) * G::TT + 64 * half;
                const unsigned dead = dead_strips[(tiles + i) % kTcMarks] >> (4 * half) & 15;
                if (warp_ok) {
                    uint32_t v0[32], v1[32];
                    tmem_ld32_nowait(ts, v0);
                    tmem_ld32_nowait(ts + 32, v1);
                    tmem_wait_ld(v0);
                    tmem_wait_ld(v1);
                    if (tok0 + 64 > d.s.ctx || dead || attn_left_out(d.s, tok0)) {   // tokens that this row does not see
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            const int t0 = tok0 + 32 * c, before = d.s.ctx - t0, all = d.s.len - t0;
                            uint32_t m = before >= 32 ? ~0u : before > 0 ? (1u << before) - 1 : 0u;
                            if (before < 32) m |= before > 0 ? (uint32_t)sees << before : -before < 64 ? (uint32_t)(sees >> -before) : 0u;
                            m &= all >= 32 ? ~0u : all > 0 ? (1u << all) - 1 : 0u;
                            if constexpr (P::SHARED) {
                                const int shared = d.s.lo - t0;
                                m &= shared >= 32 ? 0u : shared > 0 ? ~0u << shared : ~0u;
                            }
                            if ((dead >> (2 * c)) & 1) m &= 0xffff0000u;
                            if ((dead >> (2 * c + 1)) & 1) m &= 0x0000ffffu;
#pragma unroll
                            for (int x = 0; x < 32; x++)
                                if (!((m >> x) & 1)) (c ? v1 : v0)[x] = __float_as_uint(NEG);
                        }
                    }
                    float mx = NEG;
#pragma unroll
                    for (int x = 0; x < 32; x++) mx = fmaxf(mx, fmaxf(__uint_as_float(v0[x]), __uint_as_float(v1[x])));
                    const bool raise = mx * rs > top + kSlack;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float up = fmaxf(top, mx * rs);
                        const float by = up == top ? 1.f : ex2(top - up);
                        top = up;
                        sum *= by;
                        if (m > 0) {
                            if (!(ok = wait(bar_s(c + 1), ((c + 1) >> 1) & 1))) break;     // the values of the step before
                            tc_fence_after();
#pragma unroll 1
                            for (int x = 0; x < D; x += 32) {
                                uint32_t u[32];
                                tmem_ld32_nowait(to + x, u);
                                tmem_wait_ld(u);
#pragma unroll
                                for (int y = 0; y < 32; y++) u[y] = __float_as_uint(__uint_as_float(u[y]) * by);
                                tmem_st32(to + x, u);
                            }
                        }
                    }
                    const float off = kShift - (top == NEG ? 0.f : top);
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        const float a = ex2(fmaf(__uint_as_float(v0[x]), rs, off)), b = ex2(fmaf(__uint_as_float(v0[x + 1]), rs, off));
                        s0 += a; s1 += b;
                        v0[x / 2] = pack2<BF>(a, b);
                    }
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        const float a = ex2(fmaf(__uint_as_float(v1[x]), rs, off)), b = ex2(fmaf(__uint_as_float(v1[x + 1]), rs, off));
                        s0 += a; s1 += b;
                        v0[16 + x / 2] = pack2<BF>(a, b);
                    }
                    tmem_st32(ts, v0);
                    sum += s0 + s1;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p(steps + m));
            }
            if (!ok) break;
            // the last two steps' values, then both streams' maxima and sums
            steps += np;
            commits += np;
            for (int i = 0; i < 2 && ok; i++, commits++) ok = wait(bar_s(commits), (commits >> 1) & 1);
            if (!ok) break;
            ml[(st * kTcHalf + r) * 2] = top;
            ml[(st * kTcHalf + r) * 2 + 1] = sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_meet);
            if constexpr (!BF) {
                results(d);
                if (!ok) break;
            }
        }
        if constexpr (BF) cp_async_wait<0>();                                // (after a wait that gave up)
        if (tid == 0) reinterpret_cast<TcSet *>(p.counters)[blockIdx.x] = ok ? set : TcSet{};
    } else if (warp < kTcBuildWarp) {
        if constexpr (G::QUANT) regs_less<G::REGS_OTHER>();
        if (warp == kTcMmaWarp) {
            // ---------------- products ----------------
            // the whole warp walks the steps, so that operands stay in uniform registers; one lane issues
            constexpr uint32_t TYPE = BF ? 1u : 0u;
            constexpr uint32_t IDESC = (1u << 4) | (TYPE << 7) | (TYPE << 10) | ((uint32_t)(kTcHalf >> 4) << 24);
            constexpr uint32_t IDESC_S = IDESC | ((uint32_t)(G::TT >> 3) << 17), IDESC_S64 = IDESC | (64u >> 3 << 17);
            constexpr uint32_t IDESC_O = IDESC | ((uint32_t)(D >> 3) << 17) | (1u << 16);     // B N-major
            const uint64_t k_desc = sw128_desc(sb), v_desc = sw128_desc_mn(sb, G::HALF);
            const bool one = elect_one();
            int tiles = 0, pieces = 0, commits = 0, steps = 0;
            while (ok && next()) {
                if (!(ok = wait(bar_q, pieces & 1))) break;
                tc_fence_after();
                pieces++;
                const bool two = w.nq == 2;
                const int np = w.n * w.nq;
                // Scores of step m: one product of all tokens for both streams, or each stream's rows with the
                // step's 64 tokens.  Only by the elected lane.
                auto scores = [&](int m, int c, int slot) {
                    const uint32_t ds = tmem + G::S0 + 128 * (c & 1);
                    const uint64_t k = k_desc + (uint32_t)((G::OFF_RING + slot * G::TILE) >> 4);
                    if (!two) {
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            const uint32_t o = ((i >> 2) * G::HALF + (i & 3) * 32) >> 4, oq = ((i >> 2) * G::QHALF + (i & 3) * 32) >> 4;
                            umma_f16_ss(ds, k_desc + (uint32_t)((G::OFF_Q >> 4) + oq), k + o, IDESC_S, i > 0);
                        }
                    } else {
                        const uint64_t kh = k + (uint32_t)((m & 1) * (64 * 128 >> 4));
#pragma unroll
                        for (int s = 0; s < 2; s++)
#pragma unroll
                            for (int i = 0; i < D / 16; i++) {
                                const uint32_t o = ((i >> 2) * G::HALF + (i & 3) * 32) >> 4;
                                umma_f16_ss(ds + 64 * s, k_desc + (uint32_t)(((G::OFF_Q + s * G::QTILE) >> 4) + o), kh + o, IDESC_S64, i > 0);
                            }
                    }
                };
                // Lane 0 waits for the probabilities of step m, lane 1 for its values, lane 2 for the keys of
                // step m + 2 (which are there already or do not depend on step m): one test for all.
                auto wait_for = [&](int m, bool values, int slot_v, int ph_v, int slot_k, int ph_k) {
                    uint32_t bar = bar_p(steps + m), ph = (steps + m) >> 1;
                    if (lane == 1) { bar = bar_full(slot_v); ph = ph_v; }
                    if (lane == 2) { bar = bar_full(slot_k); ph = ph_k; }
                    const bool mine = (lane <= 1 && values) || (lane == 2 && slot_k >= 0);
                    bool there = !mine || mbar_try_wait_nohint(bar, ph & 1);
                    if (!__all_sync(0xffffffffu, there)) {
                        if (!there) there = mbar_wait_spin(bar, ph & 1);
                        if (!__all_sync(0xffffffffu, there)) {
                            if (lane == 0) atomicOr(error, 2);
                            return false;
                        }
                    }
                    tc_fence_after();
                    return true;
                };
                for (int m = 0; m < 2 && ok; m++) {
                    const int x = tc_k_pos<G::QUANT>(tiles, two ? 0 : m), slot = (m < np) ? x % NS : -1;
                    if (!(ok = wait_for(m, false, 0, 0, slot, x / NS))) break;
                    if (one) {
                        if (slot >= 0) scores(m, commits + m, slot);
                        umma_commit(bar_s(commits + m));
                        if (slot >= 0 && (!two || m == 1)) umma_commit(bar_empty(slot));
                    }
                    __syncwarp();
                }
                for (int m = 0; m < np && ok; m++) {
                    const int tv = two ? m >> 1 : m, tk = two ? (m + 2) >> 1 : m + 2;
                    const int xv = tc_v_pos<G::QUANT>(tiles, tv, w.n), xk = tc_k_pos<G::QUANT>(tiles, tk);
                    const int slot_v = xv % NS, slot_k = m + 2 < np ? xk % NS : -1;
                    if (!(ok = wait_for(m, true, slot_v, xv / NS, slot_k, xk / NS))) break;
                    const int c = commits + m;                               // (c + 2 has the same parity)
                    if (one) {
                        const uint64_t v = v_desc + (uint32_t)((G::OFF_RING + slot_v * G::TILE) >> 4);
#pragma unroll
                        for (int s = 0; s < G::STREAMS; s++) {
                            const uint64_t vs = v + (uint32_t)((two ? m & 1 : s) * (64 * 128 >> 4));   // 64 tokens on
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                umma_f16_ts(tmem + G::O0 + 128 * s, tmem + G::S0 + 128 * (c & 1) + 64 * s + 8 * i, vs + i * 128,
                                            IDESC_O, (m > 0 || i > 0) ? 1u : 0u);
                        }
                        if (slot_k >= 0) scores(m + 2, c, slot_k);
                        umma_commit(bar_s(c));
                        if (!two || (m & 1)) {
                            umma_commit(bar_empty(slot_v));
                            if (slot_k >= 0) umma_commit(bar_empty(slot_k));
                        }
                    }
                    __syncwarp();
                }
                commits += np + 2;
                steps += np;
                tiles += w.n;
            }
            // (every piece's last products were waited for by its softmax warps before they left)
        } else if (warp == kTcKeyWarp || warp == kTcValueWarp) {
            // ---------------- keys and values from the cache ----------------
            // a page's tokens (at most 128 of them, a box) at a time: lane i copies the tile's i-th box.  A warp for keys, one for
            // values: a box costs its warp about 100 cycles (16 of them, codes and scales of 16-token pages, 2000 per side).
            // Who waits for a slot's phase has seen the one before, as slots are emptied in the order of the positions.
            const int side = warp == kTcValueWarp;
            const int box = min(1 << p.cache.lp, G::TT), boxes = G::TT / box;
            struct Tile {
                int64_t row;            // this lane's box: its first cached row
                bool have;              // ... which exists
                unsigned valid, dead;   // boxes that exist; 16-token strips without a page
                int ctx, len, mark;     // first new token and end within the tile; mark of the piece
                int lo;                 // tokens left out
            };
            constexpr int RING = G::QUANT ? NR : NS;
            int pieces = 0, tiles = 0, lands = 0;
            int last[4] = {-1, -1, -1, -1};                                  // own positions, newest first: all that a ring can hold
            // keys or values of a tile into position x
            auto copy = [&](const Tile &q, int x) {
                const int slot = x % RING, turn = x / RING;
                if (turn && !(ok = wait(G::QUANT ? bar_rawe(slot) : bar_empty(slot), (turn - 1) & 1))) return;
                last[3] = last[2]; last[2] = last[1]; last[1] = last[0]; last[0] = x;
                if constexpr (G::QUANT) {
                    const uint32_t dst = sb + G::OFF_RAW + slot * G::RAW;
                    if (lane == 0) {
                        // tokens present, first new one (values only), page marks, mark of the piece
                        *reinterpret_cast<int4 *>(smem + G::OFF_SIDES + 16 * slot) =
                            make_int4(q.len, side ? q.ctx : G::TT, (int)q.dead | (P::SHARED ? q.lo << 8 : 0), q.mark);
                        mbar_arrive_expect_tx(bar_rawf(slot), __popc(q.valid) * box * (G::RB + 2 * G::NB));
                    }
                    __syncwarp();
                    if (q.have) {
                        bulk_g2s(dst + lane * box * G::RB, (side ? p.cache.v : p.cache.k) + q.row * G::RB, box * G::RB, bar_rawf(slot));
                        bulk_g2s(dst + G::TT * G::RB + lane * box * 2 * G::NB,
                                 (side ? p.cache.v_scale : p.cache.k_scale) + q.row * G::NB, box * 2 * G::NB, bar_rawf(slot));
                    }
                } else {
                    const uint32_t dst = sb + G::OFF_RING + slot * G::TILE;
                    const bool fix = side && (q.ctx < G::TT || q.dead || (P::SHARED && q.lo));
                    const uint32_t bar = fix ? bar_land : bar_full(slot);
                    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(q.valid) * box * G::HALVES * 128);
                    __syncwarp();
                    if (q.have)
#pragma unroll
                        for (int half = 0; half < G::HALVES; half++)
                            tma_box_2d(dst + half * G::HALF + lane * box * 128, side ? &vmap : &kmap, 64 * half, (int)q.row, bar);
                    if (fix) {
                        // zeros behind the end (stored without a look at what is there: the last tile of a short sequence is mostly that,
                        // and this warp's looking took 5 us of it) and where there is no page; new tokens' infinities and NaN out,
                        // and marked
                        if (!(ok = wait(bar_land, lands++ & 1))) return;
                        bool hit = false;
                        constexpr int N = 4;                                 // chunks at a time (G::TT * D / 8 is a multiple of 32 N)
                        const int end = (q.len * (D / 8) + 32 * N - 1) / (32 * N) * (32 * N);
#pragma unroll 4
                        for (int i = end + lane; i < G::TT * (D / 8); i += 32)
                            sts128(dst + tc_chunk<G::TT>(i / (D / 8), i % (D / 8)), make_uint4(0, 0, 0, 0));
#pragma unroll 1
                        for (int i0 = (q.dead || (P::SHARED && q.lo) ? 0 : q.ctx) * (D / 8) / (32 * N) * (32 * N) + lane; i0 < end; i0 += 32 * N) {
                            uint4 v[N];
#pragma unroll
                            for (int n = 0; n < N; n++) v[n] = lds128(dst + tc_chunk<G::TT>((i0 + 32 * n) / (D / 8), (i0 + 32 * n) % (D / 8)));
#pragma unroll
                            for (int n = 0; n < N; n++) {
                                const int r = (i0 + 32 * n) / (D / 8), c = (i0 + 32 * n) % (D / 8);
                                uint32_t u[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
                                bool any = r >= q.len || ((q.dead >> (r >> 4)) & 1) || (P::SHARED && r < q.lo);
                                if (any) {
                                    u[0] = u[1] = u[2] = u[3] = 0;
                                } else if (r >= q.ctx) {
#pragma unroll
                                    for (int y = 0; y < 4; y++) {
                                        if ((u[y] & 0x7f80u) == 0x7f80u) { u[y] &= 0xffff0000u; any = hit = true; }
                                        if ((u[y] & 0x7f800000u) == 0x7f800000u) { u[y] &= 0xffffu; any = hit = true; }
                                    }
                                }
                                if (any) sts128(dst + tc_chunk<G::TT>(r, c), make_uint4(u[0], u[1], u[2], u[3]));
                            }
                        }
                        if (hit) nan_mark[(q.mark - 1) % kTcMarks] = (uint32_t)q.mark;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_full(slot));
                    }
                }
            };
            while (ok && next()) {
                const int32_t *table = p.table + (int64_t)attn_table_row(w.s) * p.max_pages;
                auto page_of = [&](int t) {
                    const int tok = t * G::TT + lane * box;
                    return (lane < boxes && tok < w.s.len && !attn_left_out(w.s, tok + box - 1)) ? table[tok >> p.cache.lp] : -2;
                };
                int next_page = page_of(w.tile0);
                for (int t = w.tile0; t < w.tile0 + w.n && ok; t++) {
                    const int page = next_page, tok = t * G::TT + lane * box;
                    if (t + 1 < w.tile0 + w.n) next_page = page_of(t + 1);
                    Tile q;
                    q.have = page >= 0 && page < p.cache.n_pages;
                    q.row = q.have ? (((int64_t)page * p.cache.n_kv + w.h) << p.cache.lp) + (tok & ((1 << p.cache.lp) - 1)) : 0;
                    q.valid = __ballot_sync(0xffffffffu, q.have);
                    // strip i lies in box 16 i / box
                    q.dead = __ballot_sync(0xffffffffu, lane < G::TT / 16 && t * G::TT + 16 * lane < w.s.len &&
                                                            !attn_left_out(w.s, t * G::TT + 16 * lane + 15) &&
                                                            !((q.valid >> (16 * (lane & 7) / box)) & 1));
                    q.ctx = min(max(0, w.s.ctx - t * G::TT), G::TT);
                    q.len = min(w.s.len - t * G::TT, G::TT);
                    q.mark = pieces + 1;
                    q.lo = P::SHARED ? min(max(0, attn_lo(w.s) - t * G::TT), G::TT) : 0;
                    if (side == 0 && lane == 0) {
                        dead_strips[(tiles + t - w.tile0) % kTcMarks] = (uint8_t)q.dead;
                        if (q.dead) atomicOr(error, BQG_DEVERR_PAGE);
                    }
                    copy(q, side ? tc_v_pos<G::QUANT>(tiles, t - w.tile0, w.n) : tc_k_pos<G::QUANT>(tiles, t - w.tile0));
                }
                tiles += w.n;
                pieces++;
            }
            // do not leave while own copies into shared memory are in flight
            const int past = 2 * tiles + (G::QUANT ? 0 : 1);                 // the positions' end
            for (int i = 0; i < 4; i++)
                if (last[i] >= max(0, past - RING))
                    mbar_wait_spin(G::QUANT ? bar_rawf(last[i] % RING) : bar_full(last[i] % RING), (last[i] / RING) & 1);
        } else if (warp == kTcPlanWarp) {
            // ---------------- the pieces, for all roles ----------------
            // one copy of this code: a CTA's first microseconds are mostly spent on fetching instructions
            int bad = 0;
            TcWork<G::NQ, G::TT, P> work;
            work.init(p, lane, bad);
            for (int i = 0; ok; i++) {
                if (!work.next(p, w)) w.n = 0;
                if (i >= 2 && !(ok = wait(bar_pe(i), ((i >> 1) - 1) & 1))) break;
                if (lane == 0) {
                    *reinterpret_cast<TcPiece *>(smem + G::OFF_PIECES + (i & 1) * sizeof(TcPiece)) = w;
                    mbar_arrive(bar_pf(i));
                }
                __syncwarp();
                if (w.n == 0) break;
            }
            if (blockIdx.x == 0) {
                attn_check_ends(p, bad);
                if (bad) atomicOr(error, bad);
            }
        }
    } else {
        // ---------------- fp16 tiles from codes and scales ----------------
        if constexpr (G::QUANT) {
            regs_less<G::REGS_OTHER>();
            const int lt = tid - 32 * kTcBuildWarp;                          // 0 .. 255
            constexpr int STEP = 256 / G::CPT;
            const int c = lt % G::CPT, r0 = lt / G::CPT;                     // chunk c of rows r0 + i STEP
            int tiles = 0;
            auto build = [&](int x) {
                const int rs = x % NR, slot = x % NS;
                // lane 0 waits for the side, lane 1 for the slot's last products
                {
                    const uint32_t bar = lane == 0 ? bar_rawf(rs) : bar_empty(slot), ph = lane == 0 ? x / NR : x / NS - 1;
                    bool there = lane > 1 || (lane == 1 && x < NS) || mbar_try_wait_nohint(bar, ph & 1);
                    if (!__all_sync(0xffffffffu, there)) {
                        if (!there) there = mbar_wait_spin(bar, ph & 1);
                        if (!(ok = __all_sync(0xffffffffu, there))) {
                            if (lane == 0) atomicOr(error, 2);
                            return;
                        }
                    }
                }
                const int4 side = *reinterpret_cast<const int4 *>(smem + G::OFF_SIDES + 16 * rs);
                const uint32_t dst = sb + G::OFF_RING + slot * G::TILE;
                const uint8_t *src = smem + G::OFF_RAW + rs * G::RAW;
                constexpr int M = G::CHUNKS / 256;
                const bool plain = side.x >= G::TT && side.y >= G::TT && side.z == 0;
                bool hit = false;
                // STEP is a multiple of 8: a thread's chunks have the same place in their rows' swizzle.  Chunks of a row's
                // second 64 values are stored in the other order: distinct banks
                static_assert(STEP % 8 == 0, "swizzle");
                constexpr int OUT = FMT == BQG_Q8_0 ? 2 : 4;                 // chunks of fp16 from one of codes
                const int f = FMT == BQG_Q8_0 ? (c >> 2) & 1 : (c >> 1) & 1;
                uint32_t at[OUT];
#pragma unroll
                for (int k = 0; k < OUT; k++) at[k] = dst + tc_chunk<G::TT>(r0, OUT * c + (k ^ (f * (OUT / 2))));
                uint4 codes[M];
                uint32_t scale[M];
#pragma unroll
                for (int i = 0; i < M; i++) {
                    codes[i] = *reinterpret_cast<const uint4 *>(src + (i * 256 + lt) * 16);
                    scale[i] = *reinterpret_cast<const uint16_t *>(src + G::TT * G::RB + ((r0 + i * STEP) * G::NB
                                                                                           + (FMT == BQG_Q8_0 ? c >> 1 : c)) * 2);
                }
                if (!plain) {
                    // no token: zeros; a new token's scale that may leave fp16's range: its values are looked at below, and the piece marked
#pragma unroll
                    for (int i = 0; i < M; i++) {
                        const int r = r0 + i * STEP;
                        if (r >= side.x || ((side.z >> (r >> 4)) & 1) || (P::SHARED && r < side.z >> 8)) scale[i] = 0;
                        if (r >= side.y && (scale[i] & kWideScale<FMT>) == kWideScale<FMT>) hit = true;
                    }
                }
#pragma unroll
                for (int i = 0; i < M; i++) {
                    const uint4 q = codes[i];
                    const uint32_t d = __byte_perm(scale[i], 0, 0x1010), o = i * STEP * 128;
                    if constexpr (FMT == BQG_Q8_0) {
                        const uint32_t wd[4] = {f ? q.z : q.x, f ? q.w : q.y, f ? q.x : q.z, f ? q.y : q.w};
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            uint32_t u[4];
#pragma unroll
                            for (int n = 0; n < 2; n++) {
                                const uint32_t b = wd[2 * k + n] ^ 0x80808080u;
                                u[2 * n] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4140), 0x64806480u), d);
                                u[2 * n + 1] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4342), 0x64806480u), d);
                            }
                            sts128(at[k] + o, make_uint4(u[0], u[1], u[2], u[3]));
                        }
                    } else {
                        const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int k = 0; k < 4; k++) {                     // low nibbles of words 0, 1, of 2, 3, high ones
                            uint32_t u[4];
#pragma unroll
                            for (int n = 0; n < 2; n++) {
                                const uint32_t b = (wd[2 * (k & 1) + n] >> (((k >> 1) ^ f) * 4)) & 0x0f0f0f0fu;
                                u[2 * n] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4140), 0x64086408u), d);
                                u[2 * n + 1] = hmul2(hsub2(__byte_perm(b, 0x64646464u, 0x4342), 0x64086408u), d);
                            }
                            sts128(at[k] + o, make_uint4(u[0], u[1], u[2], u[3]));
                        }
                    }
                }
                if (hit) {
                    tc_drop_nonfinite<G::TT, M, OUT>(dst, r0, STEP, side.y, OUT * c);
                    nan_mark[(side.w - 1) % kTcMarks] = (uint32_t)side.w;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_rawe(rs));
                    mbar_arrive(bar_full(slot));
                }
            };
            while (ok && next()) {
                for (int t = 0; t < w.n && ok; t++) {
                    build(tc_k_pos<true>(tiles, t));
                    if (ok && t) build(tc_v_pos<true>(tiles, t - 1, w.n));
                }
                if (ok) build(tc_v_pos<true>(tiles, w.n - 1, w.n));
                tiles += w.n;
            }
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
template <int D, int ROWS, typename P = AttnParams> __global__ void __launch_bounds__(256) attn_tc_join_kernel(const P p, int ctas)
{
    pdl_wait();                              // (own_kernel relies on this order)
    pdl_launch_dependents();
    const TcSet set = reinterpret_cast<const TcSet *>(p.counters)[blockIdx.x];
    const int row = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
    if (row >= set.rows) return;
    constexpr int V = D / 32;                                                // groups of four values per warp
    const float2 *ml = reinterpret_cast<const float2 *>(p.part + (int64_t)2 * ctas * ROWS * D);
    const float4 *part = reinterpret_cast<const float4 *>(p.part);
    auto slot = [&](int c) { return attn_slot_row<1>(c, set.c0, 0); };
    // in one pass, relative to the largest maximum so far, four pieces' loads at a time
    float mt = -__builtin_huge_valf(), l = 0.f, v[4 * V];
#pragma unroll
    for (int i = 0; i < 4 * V; i++) v[i] = 0.f;
    constexpr int N = 4;
    for (int c = set.c0; c <= set.c1; c += N) {
        float2 q[N];
        float4 a[N][V];
#pragma unroll
        for (int n = 0; n < N; n++) {
            if (c + n > set.c1) break;
            q[n] = ml[slot(c + n) * ROWS + row];
#pragma unroll
            for (int i = 0; i < V; i++) a[n][i] = part[(slot(c + n) * (D / 4) + warp * V + i) * ROWS + row];
        }
#pragma unroll
        for (int n = 0; n < N; n++) {
            if (c + n > set.c1) break;
            const float up = fmaxf(mt, q[n].x);
            const float w0 = mt == up ? 1.f : ex2(mt - up), w = q[n].x == up ? 1.f : ex2(q[n].x - up);
            mt = up;
            l = l * w0 + w * q[n].y;
#pragma unroll
            for (int i = 0; i < V; i++) {
                v[4 * i] = v[4 * i] * w0 + w * a[n][i].x; v[4 * i + 1] = v[4 * i + 1] * w0 + w * a[n][i].y;
                v[4 * i + 2] = v[4 * i + 2] * w0 + w * a[n][i].z; v[4 * i + 3] = v[4 * i + 3] * w0 + w * a[n][i].w;
            }
        }
    }
    if constexpr (P::SHARED) {
        SharedSeq s{};
        s.q0 = set.q0;
        const int64_t at = shared_row(p, s, set.h, set.row0 + row);
        float4 *shared = shared_at<D>(p, at, warp * V);
        if (!p.own) {
#pragma unroll
            for (int i = 0; i < V; i++) shared[i * 32] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (warp == 0) *reinterpret_cast<float2 *>(p.rows_ml + at * 2) = make_float2(mt, l);
            return;
        }
        if (set.lo) {
            const float2 q = *reinterpret_cast<const float2 *>(p.rows_ml + at * 2);
            const float up = fmaxf(mt, q.x);
            const float a = mt == up ? 1.f : ex2(mt - up), b = q.x == up ? 1.f : ex2(q.x - up);
            l = l * a + q.y * b;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float4 f = shared[i * 32];
                v[4 * i] = v[4 * i] * a + f.x * b; v[4 * i + 1] = v[4 * i + 1] * a + f.y * b;
                v[4 * i + 2] = v[4 * i + 2] * a + f.z * b; v[4 * i + 3] = v[4 * i + 3] * a + f.w * b;
            }
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
