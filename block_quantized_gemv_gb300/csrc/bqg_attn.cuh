// bqg_attn.cuh -- attention of each sequence's newest tokens over a paged cache.
//
//   out[i, h] = sum_j p_j v_j,   p = softmax over the visible j of scale * q[i, h] . k_j
//
// The rows that share a KV head (new tokens x query heads of the group)
// share its keys and values, so a unit of work is (sequence, KV head, 64 cached
// tokens), and the floor is reading every cached row once: with few rows the
// kernel streams.  (At most 16 rows: more go to bqg_attn_tc.cuh.)
//
//  * Work is split evenly: the units of all sequences in one line (with a few of no work where a set begins, see
//    attn_kernel), each CTA a contiguous range of them, so ragged lengths and few (sequence, head)
//    pairs fill the GPU alike.  A range that begins or ends inside a
//    (sequence, head) leaves a partial result (maximum, sum,
//    unnormalised output rows) in the workspace; the CTA whose counted
//    arrival completes the set joins it, in the order of the ranges, so the
//    bits do not depend on timing.
//  * Each warp feeds itself: of a unit's 64 tokens it takes 16 (a strip, always
//    inside one page), copied with cp.async into its own ring, 16-byte
//    chunks permuted so that fragment loads meet no bank conflicts.
//    Tokens behind a sequence's end are filled with zeros, never read.
//  * The products go to the tensor cores (mma.sync m16n8k16, fp32 accumulate),
//    transposed: S^T = K Q^T with the strip's 16 tokens as the M side and tiles of 8
//    rows as N, then O^T = V^T P^T with the values as M, the tokens as K.  What a token costs
//    then grows in steps of 8 rows, and one token has few (with the rows
//    as M, 16 at least, half the products, scores, exponentials and
//    accumulators of 8 rows were padding: 637 instructions per strip).  P^T
//    goes from accumulators to operand with one movmatrix per 8 x 8.
//    bf16: as stored.  q8_0 / q4_0: a key's codes are fp16 numbers as they lie (make_q), their block sum
//    is scaled by its fp16 scale in fp32; a value's code becomes an fp16 integer (a byte under 0x64
//    is 1024 + byte) and is multiplied by the scale, rounded once to fp16 (relative 2^-11; below
//    2^-14 exact: d and so q d are multiples of 2^-24).  The queries then are fp16
//    too: each row is scaled by a power of two (exact) so that its largest
//    value lies in [1, 2), which keeps a bf16 value's eight bits down to 2^-16
//    of the largest; the power goes into the row's softmax scale.
//  * The running maximum is raised only when a score exceeds it by more than
//    kSlack (in powers of two), so the common strip needs no exchange between
//    lanes and no rescaling.  Probabilities relative to that maximum are at
//    most 2^kSlack; for fp16 they carry a factor 2^kShift, which keeps ten
//    bits down to 2^-22 of the maximum and cancels in the division.
//  * The probabilities are rounded to the values' type, since an MMA takes both operands in one: to fp16 2^-11, which does not
//    show, to bf16 2^-8 of each, as the values themselves are held.  Against 64 bits bf16 outputs are then off by 0.0023
//    (relative, root mean square); 0.0017 of that is the output's own rounding.  Two bf16 terms of a probability (2^-16 of it)
//    were tried: 0.5 to 1.5 % more time at up to 128 values and one row tile, but 3 to 5 % at 256 and with two.
//    Sums, maxima and outputs stay in fp32.
//  * Measured (head_dim 128, one new token, back to back): 32 sequences of up to 8191, 4 heads on each of 8, bf16:
//    121 us, 0.96 of the copy rate.  One of 131,071, q8_0: 56 us, 45 of them the stream, the rest the join of 57 pieces
//    per head.  8 x 4096, 32 KV heads, q4_0: 48 us against 22 for the bytes: bound by issue (59 % of the slots), as
//    one row pays for a tile of 8.  1 x 777: 8 us, latency.  Three CTAs per SM; four (128 registers)
//    spill and take 1 to 40 % longer.
#pragma once

#include "bqg_kv.cuh"

namespace bqg {

constexpr int kAttnWarps = 4;            // warps per CTA
constexpr int kStrip = 16;               // tokens per warp and unit
constexpr int kUnit = kAttnWarps * kStrip;
constexpr int kLead = 2;                 // units that beginning a set counts as, see attn_kernel
constexpr float kSlack = 6.0f;

// One sequence as the kernels work on it.
struct AttnSeq {
    int b, q0, T, ctx, len;      // first query token, new tokens, context and all cached tokens
};
// A set of tokens of a pass over shared and own tokens (SharedParams): a prefix, or a sequence without its prefix.
struct SharedSeq : AttnSeq {
    int lo;                      // tokens from here on
    int row;                     // of the block table (b: number of the set)
};
// Tokens that a set leaves out; its row of the block table.
__device__ __forceinline__ int attn_lo(const AttnSeq &) { return 0; }
__device__ __forceinline__ int attn_lo(const SharedSeq &s) { return s.lo; }
__device__ __forceinline__ bool attn_left_out(const AttnSeq &, int) { return false; }
__device__ __forceinline__ bool attn_left_out(const SharedSeq &s, int tok) { return tok < s.lo; }
__device__ __forceinline__ int attn_table_row(const AttnSeq &s) { return s.b; }
__device__ __forceinline__ int attn_table_row(const SharedSeq &s) { return s.row; }

struct AttnParams {
    using Seq = AttnSeq;
    static constexpr bool SHARED = false;
    const uint16_t *q;                   // bf16
    int64_t q_stride;
    KvCacheDev cache;
    const int32_t *table;                // [n_seq][max_pages]
    int64_t max_pages;
    const int32_t *ctx_len, *q_start;
    int n_seq;
    int64_t n_tokens;
    int max_q, n_q, group;               // group = n_q / n_kv
    const unsigned long long *mask;
    float scale_log2;                    // scale * log2(e)
    uint16_t *out;                       // bf16 [n_tokens][n_q][D]
    int *counters;                       // one per CTA, zero between calls
    float *part;                         // [2 * CTAs][rows of a tile][D], then (maximum, sum) pairs
};

// Geometry of one instantiation: RT row tiles of 8 per CTA.
template <int FMT, int D, int RT> struct AttnGeom {
    static constexpr int ROWS = 8 * RT;
    static constexpr int RB = KvRow<FMT, D>::BYTES;                     // bytes of a cached row
    static constexpr int NB = D / QK;                                   // blocks of a row
    static constexpr int CPT = RB / 16;                                 // 16-byte chunks of a row
    static constexpr int SCALES = (FMT == BQG_BF16) ? 0 : kStrip * NB * 2;
    static constexpr int STAGE = 2 * (kStrip * RB + SCALES);            // keys and values of a strip
    // strips in flight per warp, one less than stages
    static constexpr int S = (STAGE >= 4096) ? 3 : 4;
    static constexpr int KS = D / 16;                                   // MMA steps of the first product
    static constexpr bool QREG = RT * D <= 256;                         // query fragments held in registers
    static constexpr int PAD = 4;                                       // floats between merged rows: distinct banks
    static constexpr int RING = kAttnWarps * S * STAGE;
    static constexpr int MERGE = kAttnWarps * ROWS * (D + PAD) * 4;     // the ring's memory again, once drained
    static constexpr int OFF_Q = (RING > MERGE ? RING : MERGE);         // query fragments
    static constexpr int OFF_P = OFF_Q + (QREG ? 0 : RT * KS * 256);    // probabilities of the exact path
    static constexpr int OFF_ML = OFF_P + kAttnWarps * 8 * kStrip * 4;  // (maximum, sum) per warp and row
    static constexpr int OFF_VIS = OFF_ML + kAttnWarps * ROWS * 8;      // new tokens that each row sees
    static constexpr int OFF_RS = OFF_VIS + ROWS * 8;                   // softmax scale per row
    static constexpr int OFF_BIAS = OFF_RS + ROWS * 4;                  // quantized keys: [row tile][block][row], see make_q
    static constexpr int OFF_FLAG = OFF_BIAS + (FMT == BQG_BF16 ? 0 : ROWS * NB * 4);
    static constexpr int SMEM = OFF_FLAG + 16;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) { uint32_t v; asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory"); return v; }
__device__ __forceinline__ uint2 lds64(uint32_t a) { uint2 v; asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory"); return v; }
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

template <bool BF> __device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (8 x 8 of 16 bits, row lane / 4, columns 2 (lane % 4)): transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
template <bool BF> __device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) { uint32_t r; asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b)); return r; }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) { uint32_t r; asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b)); return r; }
// 2^x; results below 2^-126 are zero (a probability that far below its row's largest counts as none)
__device__ __forceinline__ float ex2(float x) { float r; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x)); return r; }

// Chunk c of token `tok` in a staged strip: the position of its 16 bytes.
// Eight consecutive tokens' chunk c, and the chunk pairs (2i, 2i + 1) of
// four consecutive tokens, lie in distinct banks.
template <int CPT> __device__ __forceinline__ uint32_t chunk_at(int tok, int c)
{
    int f;
    if constexpr (CPT >= 8) f = ((tok & 3) << 1) | ((tok >> 2) & 1);
    else if constexpr (CPT == 4) f = (tok & 2) | ((tok >> 2) & 1);
    else f = (tok >> 2) & 1;
    return (uint32_t)(tok * CPT + (c ^ f)) * 16;
}

// Whether one of 16-bit words w's two scales may take a code past fp16's range (65504), or is an infinity or NaN: from
// 512 (q8_0, |code| <= 128) or 8192 (q4_0, |code| <= 8) on, which is these exponent bits set.
template <int FMT> constexpr uint32_t kWideScale = FMT == BQG_Q8_0 ? 0x6000u : 0x7000u;
template <int FMT> __device__ __forceinline__ bool any_wide_scale(uint32_t w)
{
    constexpr uint32_t lo = kWideScale<FMT>, hi = lo << 16;
    return (w & lo) == lo || (w & hi) == hi;
}

// Sequence b with its lengths made to fit; `bad` collects BQG_DEVERR_LENGTH.
__device__ __forceinline__ AttnSeq attn_own_seq(const AttnParams &p, int b, int &bad)
{
    AttnSeq s;
    s.b = b;
    const int64_t cap = min((int64_t)0x7fff0000, p.max_pages << p.cache.lp);
    const int64_t a = p.q_start[b], e = p.q_start[b + 1], c = p.ctx_len[b];
    const int64_t q0 = min(max(a, (int64_t)0), p.n_tokens), q1 = min(max(e, q0), p.n_tokens);
    const int64_t T = min(q1 - q0, (int64_t)p.max_q);
    const int64_t ctx = min(max(c, (int64_t)0), max(cap - T, (int64_t)0));
    if (q0 != a || q1 != e || T != q1 - q0 || ctx != c || T > cap) bad |= BQG_DEVERR_LENGTH;
    s.q0 = (int)q0; s.T = (int)T; s.ctx = (int)ctx;
    s.len = (int)min(ctx + T, cap);
    return s;
}
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams &p, int b, int &bad) { return attn_own_seq(p, b, bad); }

// Attention where sequences share their first tokens.  With x the scores of a row, A its shared tokens and B its own,
//     softmax(x) v = (sum_A e^(x - m) v + sum_B e^(x - m) v) / (sum_A e^(x - m) + sum_B e^(x - m)),
// so the two sums are taken apart, each relative to a maximum of its own, and put together, in two passes.
// In the first a set is a prefix: its rows are the new tokens of all its sequences, which all
// see all of it, so its keys and values are read once for each 128 or 256 rows (up to 16: once), not once per sequence.  Its
// unnormalised rows, maxima and sums stay in the workspace in fp32.  In the second a set is a sequence without its
// prefix (attn_tc_kernel again, or for few rows bqg_own.cuh); what finishes a row adds the first pass's to it.
struct SharedParams : AttnParams {
    using Seq = SharedSeq;
    static constexpr bool SHARED = true;
    const int32_t *prefix_len, *seq_start;   // [n_prefix], [n_prefix + 1] (null: one prefix, all sequences)
    int n_prefix, n_all;                     // prefixes, sequences (n_seq: sets of this pass)
    int64_t max_shared;                      // new tokens behind one prefix at most
    int own;                                 // the second pass
    float *rows, *rows_ml;                   // unnormalised (see shared_at), (maximum, sum) pairs
};
// Prefix g: its sequences, their query tokens and the shared tokens (none where the arguments do not fit, which
// `bad` then tells: both passes come to the same answer).  A prefix that fills its row of the table does not fit where there are
// new tokens: a sequence with some has a token of its own (its last), so that its set is worked on and its rows are written.
struct SharedGroup { int s0, s1, q0, T, len; };
__device__ __forceinline__ int64_t attn_cap(const AttnParams &p) { return min((int64_t)0x7fff0000, p.max_pages << p.cache.lp); }
__device__ __forceinline__ SharedGroup shared_group(const SharedParams &p, int g, int &bad)
{
    SharedGroup r;
    const int a = p.seq_start ? p.seq_start[g] : 0, e = p.seq_start ? p.seq_start[g + 1] : p.n_all;
    r.s0 = min(max(a, 0), p.n_all);
    r.s1 = min(max(e, r.s0), p.n_all);
    const int64_t q0 = min(max((int64_t)p.q_start[r.s0], (int64_t)0), p.n_tokens);
    const int64_t q1 = min(max((int64_t)p.q_start[r.s1], q0), p.n_tokens);
    const int64_t n = p.prefix_len[g];
    const bool fits = n >= 0 && n < attn_cap(p) + (q1 == q0) && q1 - q0 <= p.max_shared;
    r.q0 = (int)q0; r.T = (int)(q1 - q0);
    r.len = fits && r.s0 < r.s1 ? (int)n : 0;
    if (r.s0 != a || r.s1 != e || (!fits && r.s0 < r.s1)) bad |= BQG_DEVERR_LENGTH;
    return r;
}
__device__ __forceinline__ SharedSeq attn_seq(const SharedParams &p, int b, int &bad)
{
    SharedSeq s;
    if (!p.own) {
        const SharedGroup g = shared_group(p, b, bad);
        s.b = b;
        s.row = g.s0;                                // its pages are the first sequence's
        s.q0 = g.q0;
        s.T = g.len ? g.T : 0;
        s.ctx = s.len = g.len;
        s.lo = 0;
        return s;
    }
    int g = 0;                                       // the last prefix that begins at b or before
    if (p.seq_start)
        for (int n = p.n_prefix; n > 1; n -= n >> 1)
            if (p.seq_start[g + (n >> 1)] <= b) g += n >> 1;
    int known = 0;                                   // (the first pass reports it)
    const SharedGroup r = shared_group(p, g, known);
    static_cast<AttnSeq &>(s) = attn_own_seq(p, b, bad);
    s.row = b;
    s.lo = r.s0 <= b && b < r.s1 ? r.len : 0;
    if (s.ctx < s.lo) {
        if (s.T) bad |= BQG_DEVERR_LENGTH;
        s.ctx = s.lo;
        s.len = (int)min((int64_t)s.lo + s.T, attn_cap(p));
    }
    return s;
}
// Number of row `row` of (set, KV head) in SharedParams::rows: a set's rows follow each other.
__device__ __forceinline__ int64_t shared_row(const SharedParams &p, const SharedSeq &s, int h, int row)
{
    return ((int64_t)h * p.n_tokens + s.q0) * p.group + row;
}
// Where values 4 i .. 4 i + 3 of it are: blocks of 32 rows, [D / 4][32][4], so that who has a row per lane (tcgen05's results) writes
// and reads 512 contiguous bytes (with whole rows, 32 lines per instruction, a small prefix's results took 6 us of its 16).
template <int D> __device__ __forceinline__ float4 *shared_at(const SharedParams &p, int64_t line, int i)
{
    return reinterpret_cast<float4 *>(p.rows) + ((line >> 5) * (D / 4) + i) * 32 + (line & 31);
}
// The set that lane `from` holds (but for its number).
__device__ __forceinline__ AttnSeq attn_shfl(const AttnSeq &s, int from)
{
    AttnSeq r;
    r.q0 = __shfl_sync(0xffffffffu, s.q0, from);
    r.T = __shfl_sync(0xffffffffu, s.T, from);
    r.ctx = __shfl_sync(0xffffffffu, s.ctx, from);
    r.len = __shfl_sync(0xffffffffu, s.len, from);
    return r;
}
__device__ __forceinline__ SharedSeq attn_shfl(const SharedSeq &s, int from)
{
    SharedSeq r;
    static_cast<AttnSeq &>(r) = attn_shfl(static_cast<const AttnSeq &>(s), from);
    r.lo = __shfl_sync(0xffffffffu, s.lo, from);
    r.row = __shfl_sync(0xffffffffu, s.row, from);
    return r;
}

// Row `row` (new token row / group, head row % group) of (sequence, KV head): its query, or null past the last.
__device__ __forceinline__ const uint16_t *attn_q_row(const AttnParams &p, const AttnSeq &s, int h, int row, int D)
{
    const int i = row / p.group, hh = row - i * p.group;
    return (i < s.T) ? p.q + (s.q0 + i) * p.q_stride + (int64_t)(h * p.group + hh) * D : nullptr;
}
// The new tokens that a row sees.
__device__ __forceinline__ unsigned long long attn_sees(const AttnParams &p, const AttnSeq &s, int row)
{
    const int i = row / p.group;
    if (i >= s.T) return 0;
    return p.mask ? p.mask[s.q0 + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
}
// a / b for a >= 0, b > 0: in 32 bits where both fit (a 64-bit division is a
// hundred dependent instructions, and several stand before a CTA's first load).
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b)
{
    if ((uint64_t)(a | b) >> 32) return a / b;
    return (int64_t)((uint32_t)a / (uint32_t)b);
}
// BQG_DEVERR_LENGTH in `bad` where the sequences together do not hold all queries (their own offsets: attn_seq).
__device__ __forceinline__ void attn_check_ends(const AttnParams &p, int &bad)
{
    if (p.q_start[0] != 0 || p.q_start[p.n_seq] != p.n_tokens) bad |= BQG_DEVERR_LENGTH;
}
__device__ __forceinline__ void attn_check_ends(const SharedParams &p, int &bad)
{
    if (p.q_start[0] != 0 || p.q_start[p.n_all] != p.n_tokens) bad |= BQG_DEVERR_LENGTH;
    if (p.seq_start && (p.seq_start[0] != 0 || p.seq_start[p.n_prefix] != p.n_all)) bad |= BQG_DEVERR_LENGTH;
}
// The units (weight(sequence) of them) of all sequences, and BQG_DEVERR_LENGTH in `bad` of some lanes; s and `mine`:
// sequence `lane` and its units.  Called by whole warps, as attn_find is, which takes them on.
template <typename P, typename W>
__device__ __forceinline__ int64_t attn_total(const P &p, int lane, W weight, int &bad, typename P::Seq &s, int64_t &mine)
{
    mine = 0;
    s = typename P::Seq{};
    if (lane < p.n_seq) {
        s = attn_seq(p, lane, bad);
        mine = weight(s);
    }
    int64_t total = mine;
    for (int b = lane + 32; b < p.n_seq; b += 32) total += weight(attn_seq(p, b, bad));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    return total;
}
// The sequence that holds number u of the line of all sequences' units; `base`: the number of its first (past u: none does).
template <typename P, typename W>
__device__ __forceinline__ typename P::Seq attn_find(const P &p, int64_t u, int lane, W weight, typename P::Seq s, int64_t mine,
                                                     int64_t &base)
{
    base = 0;
    for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
        int bad = 0;
        if (b0) {
            mine = 0;
            if (b0 + lane < p.n_seq) {
                s = attn_seq(p, b0 + lane, bad);
                mine = weight(s);
            }
        }
        int64_t sum = mine;                                                   // inclusive over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + sum > u);
        if (past) {
            const int first = __ffs(past) - 1;
            base += __shfl_sync(0xffffffffu, sum - mine, first);
            typename P::Seq r = attn_shfl(s, first);
            r.b = b0 + first;
            return r;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    base = u + 1;
    return s;
}

// A finished row: E = D / 32 values per lane, divided by their sum of weights, in bf16.
template <int E> __device__ __forceinline__ void attn_store_row(uint16_t *dst, const float (&v)[E], float sum)
{
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w[e / 2] = pack2<true>(v[e] * inv, v[e + 1] * inv);
    if constexpr (E == 2) *reinterpret_cast<uint32_t *>(dst) = w[0];
    else if constexpr (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}
// Where row `row` of CTA c's piece of a set that begins in CTA c0 lies (rows of ROWS): a CTA has at most one
// piece that a former CTA began and one that it begins and does not end.
template <int ROWS> __device__ __forceinline__ int64_t attn_slot_row(int c, int c0, int row)
{
    return (int64_t)(2 * c + (c == c0)) * ROWS + row;
}
// Rows of the pieces of CTAs c0 .. c1, joined: warp w of the CTA's takes pieces
// w, w + kAttnWarps, ... in order, the warps' results are then joined in order
// (`merged` and `ml` as in the piece itself: the caller's code behind it is the
// same).  Four pieces x four rows are in flight: what bounds this is their latency.
template <int E, int ROWS>
__device__ __forceinline__ void attn_join(const float *part, const float *part_ml, int c0, int c1, int rows, int warp, int lane,
                                          float *merged, int pitch, float *ml)
{
    constexpr int D = 32 * E, R = (E <= 4) ? 4 : 2;
    for (int r0 = 0; r0 < rows; r0 += R) {
        float v[R][E], top[R], sum[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            top[r] = -__builtin_huge_valf();
            sum[r] = 0.f;
#pragma unroll
            for (int e = 0; e < E; e++) v[r][e] = 0.f;
        }
        for (int c = c0 + warp; c <= c1; c += 4 * kAttnWarps) {
            float2 q[4][R];
            float a[4][R][E];
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const int piece = c + i * kAttnWarps;
                    q[i][r] = make_float2(-__builtin_huge_valf(), 0.f);
#pragma unroll
                    for (int e = 0; e < E; e++) a[i][r][e] = 0.f;
                    if (piece <= c1 && r0 + r < rows) {
                        const int64_t at = attn_slot_row<ROWS>(piece, c0, r0 + r);
                        q[i][r] = __ldcg(reinterpret_cast<const float2 *>(part_ml + at * 2));
                        const float *src = part + at * D + lane * E;
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            const float2 f = __ldcg(reinterpret_cast<const float2 *>(src + e));
                            a[i][r][e] = f.x; a[i][r][e + 1] = f.y;
                        }
                    }
                }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const float up = fmaxf(top[r], q[i][r].x);
                    const float old = up == top[r] ? 1.f : ex2(top[r] - up), now = up == q[i][r].x ? 1.f : ex2(q[i][r].x - up);
                    top[r] = up;
                    sum[r] = sum[r] * old + q[i][r].y * now;
#pragma unroll
                    for (int e = 0; e < E; e++) v[r][e] = v[r][e] * old + a[i][r][e] * now;
                }
        }
#pragma unroll
        for (int r = 0; r < R; r++)
            if (r0 + r < rows) {
                float *dst = merged + (warp * ROWS + r0 + r) * pitch + lane * E;
#pragma unroll
                for (int e = 0; e < E; e++) dst[e] = v[r][e];
                if (lane == 0) {
                    ml[(warp * ROWS + r0 + r) * 2] = top[r];
                    ml[(warp * ROWS + r0 + r) * 2 + 1] = sum[r];
                }
            }
    }
}

template <int FMT, int D, int RT> struct AttnKernel {
    using G = AttnGeom<FMT, D, RT>;
    static constexpr bool BF = (FMT == BQG_BF16);
    static constexpr float kShift = BF ? 0.0f : 8.0f;
    static constexpr int MT = D / 16;                         // M tiles of the second product

    // 64-token tiles of a sequence, and its units: all its rows (new tokens x heads of a group, at most ROWS) at once.
    static __device__ __forceinline__ int tiles_of(const AttnSeq &s) { return (s.len + kUnit - 1) / kUnit; }
    static __device__ __forceinline__ int64_t units(const AttnParams &p, const AttnSeq &s, int lead)
    {
        return s.T ? (int64_t)p.cache.n_kv * (tiles_of(s) + lead) : 0;
    }

    // The queries of rows row0 .. row0 + 7 as they lie (this lane: row lane / 4).  The order of the
    // values within a block follows the codes' words: q8_0 lane t = lane % 4 values
    // 8t .. 8t + 7; q4_0 values 4t .. and 16 + 4t ..
    struct RawQ { uint32_t w[D / 8]; };
    static __device__ __forceinline__ void fetch_q(const AttnParams &p, const AttnSeq &s, int h, int row0, int lane, RawQ &q)
    {
        const int t = lane & 3;
        const uint16_t *src = attn_q_row(p, s, h, row0 + (lane >> 2), D);
#pragma unroll
        for (int i = 0; i < D / 8; i++) q.w[i] = 0;
        if (!src) return;
#pragma unroll
        for (int b = 0; b < G::NB; b++) {
            if constexpr (BF) {
#pragma unroll
                for (int k = 0; k < 4; k++) q.w[4 * b + k] = *reinterpret_cast<const uint32_t *>(src + 32 * b + 8 * k + 2 * t);
            } else if constexpr (FMT == BQG_Q8_0) {
                const uint4 a = *reinterpret_cast<const uint4 *>(src + 32 * b + 8 * t);
                q.w[4 * b] = a.x; q.w[4 * b + 1] = a.y; q.w[4 * b + 2] = a.z; q.w[4 * b + 3] = a.w;
            } else {
                const uint2 a = *reinterpret_cast<const uint2 *>(src + 32 * b + 4 * t);
                const uint2 c = *reinterpret_cast<const uint2 *>(src + 32 * b + 16 + 4 * t);
                q.w[4 * b] = a.x; q.w[4 * b + 1] = a.y; q.w[4 * b + 2] = c.x; q.w[4 * b + 3] = c.y;
            }
        }
    }
    // Their fragments (KS steps x 2 registers), the softmax scale of this lane's row, and bias[b]:
    // a code's bits are taken as an fp16 number as they lie, u 2^-24 exactly for the unsigned code u = q + B, so
    //     sum q_k = 2^24 (sum u 2^-24 q_k  -  B 2^-24 sum q_k),
    // whose second term is what the products of block b begin with.  (q4_0's nibbles 2, 3 of a half word are 16 u 2^-24: their
    // queries are smaller by 16.)
    static __device__ __forceinline__ void make_q(const AttnParams &p, const RawQ &q, uint32_t (&qf)[G::KS][2], float &rs,
                                                  float (&bias)[G::NB])
    {
        rs = p.scale_log2;
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < D / 8; i++) qf[i >> 1][i & 1] = q.w[i];
        } else {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; i++) top = fmaxf(top, fmaxf(fabsf(bf16_lo(q.w[i])), fabsf(bf16_hi(q.w[i]))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float inv = 1.f;
            if (top > 0.f && top < __int_as_float(0x7f800000)) {
                const uint32_t ex = min(__float_as_uint(top) >> 23, 253u);
                inv = __uint_as_float((254u - ex) << 23);                       // 2^(127 - ex)
                rs = fmaxf(p.scale_log2 * (1.0f / inv), 1.17549435e-38f);       // 1 / inv: a power of two
            }
#pragma unroll
            for (int b = 0; b < G::NB; b++) {
                uint32_t w[4] = {q.w[4 * b], q.w[4 * b + 1], q.w[4 * b + 2], q.w[4 * b + 3]};
                if constexpr (FMT == BQG_Q4_0) {                                // even values first
                    const uint32_t a = w[0], c = w[2];
                    w[0] = __byte_perm(a, w[1], 0x5410); w[1] = __byte_perm(a, w[1], 0x7632);
                    w[2] = __byte_perm(c, w[3], 0x5410); w[3] = __byte_perm(c, w[3], 0x7632);
                }
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float by = (j >> 1) || FMT == BQG_Q8_0 ? 1.0f : 16.0f;     // (16 inv may be infinite)
                    qf[2 * b + (j >> 1)][j & 1] = pack2<false>(bf16_lo(w[j]) * inv * by, bf16_hi(w[j]) * inv * by);
                }
                float part[2] = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&qf[2 * b + (j >> 1)][j & 1]));
                    part[j >> 1] += f.x + f.y;
                }
                float sum = FMT == BQG_Q8_0 ? part[0] + part[1] : fmaf(16.0f, part[1], part[0]);
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                bias[b] = sum * (FMT == BQG_Q8_0 ? -0x1p-17f : -0x1p-21f);      // 128 2^-24, 8 2^-24
            }
        }
    }

    // Copies of strip tokens tok0 .. tok0 + 15 of (sequence, head) into `st`; ok: the page is in the cache.
    template <typename Seq>
    static __device__ __forceinline__ void issue(const AttnParams &p, const Seq &s, int h, int tok0, int page, bool ok,
                                                 uint32_t st, int lane)
    {
        const int at = tok0 & ((1 << p.cache.lp) - 1);
        const int64_t row = ok ? ((((int64_t)page * p.cache.n_kv + h) << p.cache.lp) + at) : 0;
        const int n = ok ? s.len - tok0 : 0;                                     // tokens to fetch, if under 16
        const uint8_t *k = p.cache.k + row * G::RB + lane * 16, *v = p.cache.v + row * G::RB + lane * 16;
        constexpr int CH = BF ? 1 : G::SCALES / 16;                              // chunks of one side's scales
        const uint8_t *sc = nullptr;
        if constexpr (!BF)
            sc = reinterpret_cast<const uint8_t *>((lane < CH ? p.cache.k_scale : p.cache.v_scale) + row * G::NB) + lane % CH * 16;
        if (n >= kStrip && !attn_left_out(s, tok0)) {
#pragma unroll
            for (int i = 0; i < G::CPT / 2; i++) {
                const uint32_t d = st + chunk_at<G::CPT>((i * 32 + lane) / G::CPT, lane % G::CPT);
                cp_async16(d, k + i * 512, 16);
                cp_async16(d + kStrip * G::RB, v + i * 512, 16);
            }
            if constexpr (!BF)
                if (lane < 2 * CH) cp_async16(st + 2 * kStrip * G::RB + lane * 16, sc, 16);
        } else {                                                                 // zeros behind the end, and for tokens left out
#pragma unroll
            for (int i = 0; i < G::CPT / 2; i++) {
                const int tok = (i * 32 + lane) / G::CPT;
                const uint32_t d = st + chunk_at<G::CPT>(tok, lane % G::CPT);
                const int bytes = tok < n && !attn_left_out(s, tok0 + tok) ? 16 : 0;
                cp_async16(d, bytes ? k + i * 512 : p.cache.k, bytes);
                cp_async16(d + kStrip * G::RB, bytes ? v + i * 512 : p.cache.v, bytes);
            }
            if constexpr (!BF)
                if (lane < 2 * CH) {
                    const int bytes = min(max(n * G::NB * 2 - lane % CH * 16, 0), 16);
                    cp_async16(st + 2 * kStrip * G::RB + lane * 16, bytes ? sc : reinterpret_cast<const uint8_t *>(p.cache.k_scale), bytes);
                }
        }
    }

    // Scores of the strip in stage `st`: s[row tile] = tokens lane / 4 (elements 0, 1) and 8 on (2, 3) x
    // rows 2 (lane % 4) and the next.
    // bias: this lane's part of the row tiles' OFF_BIAS.
    template <typename QF>
    static __device__ __forceinline__ void scores(uint32_t st, int lane, const QF &qf, uint32_t bias, float (&s)[RT][4])
    {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int m = 0; m < RT; m++)
#pragma unroll
            for (int i = 0; i < 4; i++) s[m][i] = 0.f;
        if constexpr (BF) {
            const int tok = lane & 15, hi = lane >> 4;
#pragma unroll
            for (int ks = 0; ks < G::KS; ks++) {
                uint32_t a[4];
                ldsm_x4(st + chunk_at<G::CPT>(tok, 2 * ks + hi), a);
#pragma unroll
                for (int m = 0; m < RT; m++) {
                    uint32_t b[2];
                    qf.get(m, ks, b);
                    mma16816<true>(s[m], a, b[0], b[1]);
                }
            }
        } else {
            const uint32_t sc = st + 2 * kStrip * G::RB;
            uint32_t dw[2][G::NB / 2];                   // scales of tokens g and g + 8
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const uint32_t at = sc + (8 * x + g) * G::NB * 2;
                if constexpr (G::NB == 2) {
                    dw[x][0] = lds32(at);
                } else {
#pragma unroll
                    for (int i = 0; i < G::NB / 2; i += 2) {
                        const uint2 v = lds64(at + 4 * i);
                        dw[x][i] = v.x; dw[x][i + 1] = v.y;
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < G::NB; b++) {
                uint32_t e[2][4];                        // of tokens g, g + 8: the operand's value pairs, MMA 0 then 1
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    if constexpr (FMT == BQG_Q8_0) {
                        uint2 w = lds64(st + chunk_at<G::CPT>(8 * x + g, 2 * b + (t >> 1)) + (t & 1) * 8);
                        w.x ^= 0x80808080u; w.y ^= 0x80808080u;              // q + 128
                        e[x][0] = __byte_perm(w.x, 0, 0x4140);
                        e[x][1] = __byte_perm(w.x, 0, 0x4342);
                        e[x][2] = __byte_perm(w.y, 0, 0x4140);
                        e[x][3] = __byte_perm(w.y, 0, 0x4342);
                    } else {
                        const uint32_t w = lds32(st + chunk_at<G::CPT>(8 * x + g, b) + t * 4), w8 = w >> 8;
                        e[x][0] = w & 0x000f000fu;
                        e[x][1] = w8 & 0x000f000fu;
                        e[x][2] = w & 0x00f000f0u;
                        e[x][3] = w8 & 0x00f000f0u;
                    }
                }
                const uint32_t h0 = dw[0][b >> 1], h1 = dw[1][b >> 1];
                const float d0 = half_bits_to_float((b & 1) ? h0 >> 16 : h0 & 0xffffu);
                const float d1 = half_bits_to_float((b & 1) ? h1 >> 16 : h1 & 0xffffu);
                const uint32_t a0[4] = {e[0][0], e[1][0], e[0][1], e[1][1]}, a1[4] = {e[0][2], e[1][2], e[0][3], e[1][3]};
#pragma unroll
                for (int m = 0; m < RT; m++) {
                    const uint2 c = lds64(bias + (m * G::NB + b) * 32);
                    float acc[4] = {__uint_as_float(c.x), __uint_as_float(c.y), __uint_as_float(c.x), __uint_as_float(c.y)};
                    uint32_t q[2];
                    qf.get(m, 2 * b, q);
                    mma16816<false>(acc, a0, q[0], q[1]);
                    qf.get(m, 2 * b + 1, q);
                    mma16816<false>(acc, a1, q[0], q[1]);
                    s[m][0] = fmaf(acc[0], d0, s[m][0]);
                    s[m][1] = fmaf(acc[1], d0, s[m][1]);
                    s[m][2] = fmaf(acc[2], d1, s[m][2]);
                    s[m][3] = fmaf(acc[3], d1, s[m][3]);
                }
            }
#pragma unroll
            for (int m = 0; m < RT; m++)
#pragma unroll
                for (int i = 0; i < 4; i++) s[m][i] *= FMT == BQG_Q8_0 ? 0x1p24f : 0x1p20f;
        }
    }

    // o += V^T P^T for the strip in stage `st`.
    static __device__ __forceinline__ void add_values(uint32_t st, int lane, const uint32_t (&pb)[RT][2], float (&o)[RT][MT][4])
    {
        const int t = lane & 3;
        const uint32_t vst = st + kStrip * G::RB;
        const int tok = lane & 15, hi = lane >> 4;       // ldmatrix rows: tokens 0..15 of chunk c, then of c + 1
        if constexpr (BF) {
#pragma unroll
            for (int n = 0; n < MT; n++) {
                uint32_t r[4];
                ldsm_x4_trans(vst + chunk_at<G::CPT>(tok, 2 * n + hi), r);
                const uint32_t a[4] = {r[0], r[2], r[1], r[3]};
#pragma unroll
                for (int m = 0; m < RT; m++) mma16816<true>(o[m][n], a, pb[m][0], pb[m][1]);
            }
        } else {
            const uint32_t sc = st + 2 * kStrip * G::RB + G::SCALES;
            uint32_t dw[2][G::NB];                       // scales of tokens 8x + 2t and 8x + 2t + 1
#pragma unroll
            for (int x = 0; x < 2; x++)
#pragma unroll
                for (int i = 0; i < G::NB; i += 2) {
                    const uint2 v = lds64(sc + ((8 * x + 2 * t) * G::NB + 2 * i) * 2);
                    dw[x][i] = v.x; dw[x][i + 1] = v.y;
                }
            auto pair = [&](int x, int b) {              // (scale of token 8x + 2t, of 8x + 2t + 1) of block b
                return __byte_perm(dw[x][b >> 1], dw[x][(G::NB + b) >> 1], (b & 1) ? 0x7632 : 0x5410);
            };
            // sixteen values, the even ones as the tile's rows 0..7, the odd ones as 8..15: word lo of tokens 0..7,
            // up of 8..15, one biased code per byte
            auto tile = [&](int n, uint32_t lo, uint32_t up, uint32_t bias, uint32_t s0, uint32_t s1) {
                const uint32_t a[4] = {hmul2(hsub2(__byte_perm(lo, 0x64646464u, 0x4240), bias), s0),
                                       hmul2(hsub2(__byte_perm(lo, 0x64646464u, 0x4341), bias), s0),
                                       hmul2(hsub2(__byte_perm(up, 0x64646464u, 0x4240), bias), s1),
                                       hmul2(hsub2(__byte_perm(up, 0x64646464u, 0x4341), bias), s1)};
#pragma unroll
                for (int m = 0; m < RT; m++) mma16816<false>(o[m][n], a, pb[m][0], pb[m][1]);
            };
            if constexpr (FMT == BQG_Q8_0) {
#pragma unroll
                for (int b = 0; b < G::NB; b++) {
                    uint32_t r[4];
                    ldsm_x4_trans(vst + chunk_at<G::CPT>(tok, 2 * b + hi), r);
                    const uint32_t s0 = pair(0, b), s1 = pair(1, b);
                    tile(2 * b, r[0] ^ 0x80808080u, r[1] ^ 0x80808080u, 0x64806480u, s0, s1);
                    tile(2 * b + 1, r[2] ^ 0x80808080u, r[3] ^ 0x80808080u, 0x64806480u, s0, s1);
                }
            } else {
#pragma unroll
                for (int b = 0; b < G::NB; b += 2) {
                    uint32_t r[4];
                    ldsm_x4_trans(vst + chunk_at<G::CPT>(tok, b + hi), r);
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const uint32_t s0 = pair(0, b + j), s1 = pair(1, b + j);
                        tile(2 * (b + j), r[2 * j] & 0x0f0f0f0fu, r[2 * j + 1] & 0x0f0f0f0fu, 0x64086408u, s0, s1);
                        tile(2 * (b + j) + 1, (r[2 * j] >> 4) & 0x0f0f0f0fu, (r[2 * j + 1] >> 4) & 0x0f0f0f0fu, 0x64086408u, s0, s1);
                    }
                }
            }
        }
    }

    // The output's value that row g (hi: g + 8) of M tile n is.
    static __device__ __forceinline__ int dim_of(int n, int g, int hi) { return BF ? 16 * n + 8 * hi + g : 16 * n + 2 * g + hi; }
    // Value `dim` of token `tok` of the staged strip, in fp32.
    static __device__ __forceinline__ float value_of(uint32_t st, int tok, int dim)
    {
        const uint32_t vst = st + kStrip * G::RB;
        if constexpr (BF) {
            const uint32_t w = lds32(vst + chunk_at<G::CPT>(tok, dim / 8) + (dim % 8) / 2 * 4);
            return (dim & 1) ? bf16_hi(w) : bf16_lo(w);
        } else {
            const uint32_t sa = st + 2 * kStrip * G::RB + G::SCALES + (tok * G::NB + (dim / QK & ~1)) * 2;
            const uint32_t dw = lds32(sa);
            const float d = half_bits_to_float((dim / QK & 1) ? dw >> 16 : dw & 0xffffu);
            const int byte = (FMT == BQG_Q8_0) ? dim : dim / QK * 16 + dim % 16;
            const uint32_t w = lds32(vst + chunk_at<G::CPT>(tok, byte / 16) + (byte % 16) / 4 * 4) >> (8 * (byte % 4));
            if constexpr (FMT == BQG_Q8_0) return (float)(int8_t)(w & 0xffu) * d;
            else return (float)((int)((dim % QK < 16 ? w : w >> 4) & 15u) - 8) * d;
        }
    }
    // Some value of the staged strip may be an infinity or NaN, as it is or in fp16 (the same answer in every lane).
    static __device__ __forceinline__ bool any_nonfinite(uint32_t st, int lane)
    {
        bool bad = false;
        if constexpr (BF) {
#pragma unroll 1
            for (int i = lane; i < kStrip * G::RB / 4; i += 32) {
                const uint32_t w = lds32(st + kStrip * G::RB + 4 * i);
                bad |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
            }
        } else {
#pragma unroll 1
            for (int i = lane; i < G::SCALES / 4; i += 32) {
                const uint32_t w = lds32(st + 2 * kStrip * G::RB + G::SCALES + 4 * i);
                bad |= any_wide_scale<FMT>(w);
            }
        }
        return __any_sync(0xffffffffu, bad);
    }
    // The staged strip's first n tokens are left out, and their codes zeros (issue): zeros for their values' scales, of which 16 bytes
    // belong to several tokens and come together.
    static __device__ __forceinline__ void leave_out(uint32_t st, int n, int lane)
    {
        if constexpr (!BF) {
#pragma unroll 1
            for (int i = lane; i < n * (G::NB / 2); i += 32) sts32(st + 2 * kStrip * G::RB + G::SCALES + 4 * i, 0);
            __syncwarp();
        }
    }

    // What a warp has of its rows (this lane: 8 m + 2 t and the next): outputs and their maximum and sum so far.
    struct Rows {
        float o[RT][MT][4], top[RT][2], sum[RT][2], from[RT][2], rs[RT][2];   // from: what the exponents are relative to; softmax scale
        __device__ __forceinline__ void begin(const float *row_scale, int t)
        {
#pragma unroll
            for (int m = 0; m < RT; m++) {
                rs[m][0] = row_scale[8 * m + 2 * t];
                rs[m][1] = row_scale[8 * m + 2 * t + 1];
                top[m][0] = top[m][1] = -__builtin_huge_valf();
                sum[m][0] = sum[m][1] = 0.f;
                from[m][0] = from[m][1] = kShift;
#pragma unroll
                for (int x = 0; x < MT; x++)
#pragma unroll
                    for (int i = 0; i < 4; i++) o[m][x][i] = 0.f;
            }
        }
    };
    // The strip in stage `st`, tokens tok0 .. of s, into w; ok: its page is in the cache.  bias: this lane's part of the row
    // tiles' biases (make_q); row_sees: the new tokens that each row sees; pw: room for the probabilities of the exact path.
    template <typename QF, typename Seq>
    static __device__ __forceinline__ void strip(uint32_t st, int lane, const QF &qf, uint32_t bias, const unsigned long long *row_sees,
                                                 const Seq &s, int tok0, bool ok, float *pw, Rows &w)
    {
        constexpr float NEG = -__builtin_huge_valf();
        const int g = lane >> 2, t = lane & 3;
        float sc[RT][4];
        scores(st, lane, qf, bias, sc);
        const bool edge = tok0 + kStrip > s.ctx || !ok || attn_left_out(s, tok0);   // new tokens, the end, no page, shared ones
        if (edge) {
#pragma unroll
            for (int m = 0; m < RT; m++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const unsigned long long sees = row_sees[8 * m + 2 * t + r];
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const int tok = tok0 + 8 * x + g;
                        const bool see = ok && !attn_left_out(s, tok) && (tok < s.ctx || (tok < s.len && ((sees >> (tok - s.ctx)) & 1)));
                        if (!see) sc[m][2 * x + r] = NEG;
                    }
                }
        }
        // raise the running maximum where a score is well above it
        bool raise = false;
#pragma unroll
        for (int m = 0; m < RT; m++)
#pragma unroll
            for (int r = 0; r < 2; r++) raise |= fmaxf(sc[m][r], sc[m][2 + r]) * w.rs[m][r] > w.top[m][r] + kSlack;
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int m = 0; m < RT; m++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    float v = fmaxf(sc[m][r], sc[m][2 + r]) * w.rs[m][r];
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    v = fmaxf(v, w.top[m][r]);
                    const float c = (v == w.top[m][r]) ? 1.f : ex2(w.top[m][r] - v);
                    w.top[m][r] = v;
                    w.from[m][r] = kShift - (v == NEG ? 0.f : v);
                    w.sum[m][r] *= c;
#pragma unroll
                    for (int x = 0; x < MT; x++) { w.o[m][x][r] *= c; w.o[m][x][2 + r] *= c; }
                }
        }
        uint32_t pb[RT][2];
        const bool exact = edge && any_nonfinite(st, lane);
#pragma unroll
        for (int m = 0; m < RT; m++) {
            float e[4];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                e[r] = ex2(fmaf(sc[m][r], w.rs[m][r], w.from[m][r]));
                e[2 + r] = ex2(fmaf(sc[m][2 + r], w.rs[m][r], w.from[m][r]));
                w.sum[m][r] += e[r] + e[2 + r];
            }
            pb[m][0] = transpose8x8(pack2<BF>(e[0], e[1]));
            pb[m][1] = transpose8x8(pack2<BF>(e[2], e[3]));
            if (exact) {
                // an infinity or NaN (or a value that is one in fp16) among tokens that some rows do not see:
                // 0 x inf must not reach them, so this strip's products are taken one by one in fp32
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; i++) pw[(8 * (i >> 1) + g) * 8 + 2 * t + (i & 1)] = sc[m][i] == NEG ? -1.f : e[i];
                __syncwarp();
#pragma unroll 1
                for (int k = 0; k < kStrip; k++) {
                    const float p0 = pw[k * 8 + 2 * t], p1 = pw[k * 8 + 2 * t + 1];
#pragma unroll
                    for (int x = 0; x < MT; x++)
#pragma unroll
                        for (int hi = 0; hi < 2; hi++) {
                            const float v = value_of(st, k, dim_of(x, g, hi));
                            if (!(p0 < 0.f)) w.o[m][x][2 * hi] = fmaf(p0, v, w.o[m][x][2 * hi]);
                            if (!(p1 < 0.f)) w.o[m][x][2 * hi + 1] = fmaf(p1, v, w.o[m][x][2 * hi + 1]);
                        }
                }
            }
        }
        if (!exact) add_values(st, lane, pb, w.o);
    }
};

// Query fragments in registers, or shared by the CTA's warps in shared memory.
template <int RT, int KS> struct QRegs {
    uint32_t f[RT][KS][2];
    __device__ __forceinline__ void get(int m, int ks, uint32_t (&b)[2]) const { b[0] = f[m][ks][0]; b[1] = f[m][ks][1]; }
};
template <int RT, int KS> struct QShared {
    uint32_t addr;      // this lane's 8 bytes of fragment (0, 0)
    __device__ __forceinline__ void get(int m, int ks, uint32_t (&b)[2]) const
    {
        const uint2 v = lds64(addr + (m * KS + ks) * 256);
        b[0] = v.x; b[1] = v.y;
    }
};

template <int FMT, int D, int RT, typename P = AttnParams>
__global__ void __launch_bounds__(32 * kAttnWarps) attn_kernel(const P p, int *error)
{
    using Seq = typename P::Seq;
    using G = AttnGeom<FMT, D, RT>;
    using A = AttnKernel<FMT, D, RT>;
    constexpr int S = G::S, MT = A::MT;
    constexpr float NEG = -__builtin_huge_valf();
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    float *const ml = reinterpret_cast<float *>(smem + G::OFF_ML);            // [warp][row][2]
    float *const row_scale = reinterpret_cast<float *>(smem + G::OFF_RS);
    float *const row_bias = reinterpret_cast<float *>(smem + G::OFF_BIAS);
    unsigned long long *const row_sees = reinterpret_cast<unsigned long long *>(smem + G::OFF_VIS);
    float *const merged = reinterpret_cast<float *>(smem);                    // [warp][row][D + PAD]
    pdl_wait();                              // (own_kernel relies on this order)
    pdl_launch_dependents();

    // This CTA's range of units.  Where there may be half as many sets (sequence, KV head) as CTAs, CTAs
    // with several sets' pieces would be last: a piece's start and end cost 3 to 4 us, so each set begins with
    // kLead units that are no work.  Measured over 2 to 200 sequences of 60 to 3000 tokens, 8 KV heads, q8_0 and bf16, against none:
    // with 2 on average 0.94 of the time, at most 1.05 (200 of 1000 tokens, bf16: 91 us against 103); with 4 0.95, but up to 1.33
    // for short contexts.  With fewer sets a CTA has one piece or is near it, and its range is better left as it is.
    int bad = 0;
    const int lead = 2 * (int64_t)p.n_seq * p.cache.n_kv >= gridDim.x ? kLead : 0;
    auto weight = [&](const Seq &q) { return A::units(p, q, lead); };
    int64_t mine;
    Seq s;
    const int64_t total = attn_total(p, lane, weight, bad, s, mine);
    if (blockIdx.x == 0 && warp == 0) {
        attn_check_ends(p, bad);
        if (bad) atomicOr(error, bad);
    }
    const int64_t per = div_pos(total + gridDim.x - 1, gridDim.x);
    int64_t u = per * blockIdx.x;
    const int64_t u_end = min(u + per, total);
    if (u >= u_end) return;
    int64_t base;
    s = attn_find(p, u, lane, weight, s, mine, base);
    int pages_bad = 0;

    while (u < u_end) {
        while (u - base >= A::units(p, s, lead)) {                            // next sequence with work
            base += A::units(p, s, lead);
            s = attn_seq(p, s.b + 1, bad);
        }
        const int64_t off = u - base;
        const int tiles = A::tiles_of(s);
        const int h = (int)div_pos(off, tiles + lead), first = (int)(off - (int64_t)h * (tiles + lead));
        const int take = (int)min((int64_t)(tiles + lead - first), u_end - u);
        const int tile0 = max(first - lead, 0), n = first + take - lead - tile0;   // units of this piece
        if (n <= 0) {
            u += take;
            continue;
        }
        const int64_t seg0 = u - first + lead;                                // first unit of the whole (sequence, head)
        const int rows = s.T * p.group;

        // strips of this warp: tokens 64 (tile0 + j) + 16 warp ..
        const uint32_t ring = sb + warp * S * G::STAGE;
        const int32_t *table = p.table + (int64_t)attn_table_row(s) * p.max_pages;
        // pages of the warp's strips j0 .. j0 + 31, one per lane
        auto pages_from = [&](int j0) {
            const int tok0 = (tile0 + j0 + lane) * kUnit + warp * kStrip;
            return (j0 + lane < n && tok0 < s.len) ? table[tok0 >> p.cache.lp] : -1;
        };
        int pages = pages_from(0);
        // queries (their loads are under way when the first strips are requested)
        std::conditional_t<G::QREG, QRegs<RT, G::KS>, QShared<RT, G::KS>> qf;
        typename A::RawQ raw[G::QREG ? RT : 1];
        if constexpr (G::QREG) {
#pragma unroll
            for (int m = 0; m < RT; m++) A::fetch_q(p, s, h, 8 * m, lane, raw[m]);
        } else if (warp < RT) {
            A::fetch_q(p, s, h, 8 * warp, lane, raw[0]);
        }
        unsigned valid = 0;                                                   // stages whose page is in the cache
        auto issue = [&](int j, int st) {
            const int tok0 = (tile0 + j) * kUnit + warp * kStrip;
            const int page = __shfl_sync(0xffffffffu, pages, j & 31);
            valid &= ~(1u << st);
            if (j < n && tok0 < s.len) {
                const bool ok = page >= 0 && page < p.cache.n_pages;
                if (!ok) pages_bad = BQG_DEVERR_PAGE;
                valid |= (unsigned)ok << st;
                A::issue(p, s, h, tok0, page, ok, ring + st * G::STAGE, lane);
            }
            cp_async_commit();
            if ((j & 31) == 31) pages = pages_from(j + 1);
        };
#pragma unroll 1
        for (int j = 0; j < S - 1; j++) issue(j, j);

        // the queries' fragments, and what their rows see
        if constexpr (G::QREG) {
#pragma unroll
            for (int m = 0; m < RT; m++) {
                float r;
                float bias[G::NB];
                A::make_q(p, raw[m], qf.f[m], r, bias);
                if (warp == 0 && t == 0) {
                    row_scale[8 * m + g] = r;
                    if constexpr (!A::BF)
#pragma unroll
                        for (int b = 0; b < G::NB; b++) row_bias[(m * G::NB + b) * 8 + g] = bias[b];
                }
            }
        } else {
            static_assert(G::QREG || RT <= kAttnWarps, "a row tile per warp");
            qf.addr = sb + G::OFF_Q + lane * 8;
            if (warp < RT) {
                uint32_t f[G::KS][2];
                float r;
                float bias[G::NB];
                A::make_q(p, raw[0], f, r, bias);
#pragma unroll
                for (int ks = 0; ks < G::KS; ks++)
                    *reinterpret_cast<uint2 *>(smem + G::OFF_Q + (warp * G::KS + ks) * 256 + lane * 8) = make_uint2(f[ks][0], f[ks][1]);
                if (t == 0) {
                    row_scale[8 * warp + g] = r;
                    if constexpr (!A::BF)
#pragma unroll
                        for (int b = 0; b < G::NB; b++) row_bias[(warp * G::NB + b) * 8 + g] = bias[b];
                }
            }
        }
        if (tid < G::ROWS) row_sees[tid] = attn_sees(p, s, tid);
        __syncthreads();
        typename A::Rows r;
        r.begin(row_scale, t);

        int stage = 0;                                                        // j % S
#pragma unroll 1
        for (int j = 0; j < n; j++) {
            cp_async_wait<S - 2>();
            __syncwarp();
            issue(j + S - 1, stage ? stage - 1 : S - 1);
            const int tok0 = (tile0 + j) * kUnit + warp * kStrip;
            if (tok0 >= s.len) break;
            const uint32_t st = ring + stage * G::STAGE;
            const bool ok = (valid >> stage) & 1;
            stage = stage + 1 == S ? 0 : stage + 1;
            A::strip(st, lane, qf, sb + G::OFF_BIAS + t * 8, row_sees, s, tok0, ok,
                     reinterpret_cast<float *>(smem + G::OFF_P) + warp * 8 * kStrip, r);
        }
        cp_async_wait<0>();
        __syncthreads();                                                      // the ring's memory is free

        // the four warps' results of this piece, joined
#pragma unroll
        for (int m = 0; m < RT; m++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                r.sum[m][i] += __shfl_xor_sync(0xffffffffu, r.sum[m][i], 4);
                r.sum[m][i] += __shfl_xor_sync(0xffffffffu, r.sum[m][i], 8);
                r.sum[m][i] += __shfl_xor_sync(0xffffffffu, r.sum[m][i], 16);
                const int row = 8 * m + 2 * t + i;
                if (g == 0) {
                    ml[(warp * G::ROWS + row) * 2] = r.top[m][i];
                    ml[(warp * G::ROWS + row) * 2 + 1] = r.sum[m][i];
                }
                float *dst = merged + (warp * G::ROWS + row) * (D + G::PAD);
#pragma unroll
                for (int x = 0; x < MT; x++) {
                    if constexpr (A::BF) {
                        dst[16 * x + g] = r.o[m][x][i];
                        dst[16 * x + 8 + g] = r.o[m][x][2 + i];
                    } else {
                        *reinterpret_cast<float2 *>(dst + 16 * x + 2 * g) = make_float2(r.o[m][x][i], r.o[m][x][2 + i]);
                    }
                }
            }
        __syncthreads();
        const int c0 = (int)div_pos(seg0, per), c1 = (int)div_pos(seg0 + tiles - 1, per);  // CTAs that share the segment
        const int cta = (int)blockIdx.x;
        constexpr int E = D / 32;                                             // values per lane of a row
        float *const part_ml = p.part + (int64_t)2 * gridDim.x * G::ROWS * D;
        auto out_row = [&](int row) {
            const int i = row / p.group, hh = row - i * p.group;
            return p.out + ((int64_t)(s.q0 + i) * p.n_q + h * p.group + hh) * D + lane * E;
        };
        // rows of `merged`, the warps' results joined: into the output, or the workspace
        auto finish = [&](bool last) {
            for (int row = warp; row < rows; row += kAttnWarps) {
                float mt = NEG;
#pragma unroll
                for (int w = 0; w < kAttnWarps; w++) mt = fmaxf(mt, ml[(w * G::ROWS + row) * 2]);
                float v[E], l = 0.f;
#pragma unroll
                for (int e = 0; e < E; e++) v[e] = 0.f;
#pragma unroll
                for (int w = 0; w < kAttnWarps; w++) {
                    const float mw = ml[(w * G::ROWS + row) * 2];
                    const float c = (mw == mt) ? 1.f : ex2(mw - mt);
                    l += c * ml[(w * G::ROWS + row) * 2 + 1];
                    const float *src = merged + (w * G::ROWS + row) * (D + G::PAD) + lane * E;
#pragma unroll
                    for (int e = 0; e < E; e++) v[e] += c * src[e];
                }
                if (last) {
                    if constexpr (P::SHARED) {                                // a prefix: for the second pass
                        const int64_t at = shared_row(p, s, h, row);
                        if constexpr (E == 2) {
                            reinterpret_cast<float2 *>(shared_at<D>(p, at, lane >> 1))[lane & 1] = make_float2(v[0], v[1]);
                        } else {
#pragma unroll
                            for (int e = 0; e < E; e += 4)
                                *shared_at<D>(p, at, (lane * E + e) / 4) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        }
                        if (lane == 0) *reinterpret_cast<float2 *>(p.rows_ml + at * 2) = make_float2(mt, l);
                        continue;
                    }
                    attn_store_row<E>(out_row(row), v, l);
                } else {
                    const int64_t at = attn_slot_row<G::ROWS>(cta, c0, row);
                    float *dst = p.part + at * D + lane * E;
#pragma unroll
                    for (int e = 0; e < E; e += 2) *reinterpret_cast<float2 *>(dst + e) = make_float2(v[e], v[e + 1]);
                    if (lane == 0) *reinterpret_cast<float2 *>(part_ml + at * 2) = make_float2(mt, l);
                }
            }
        };
        finish(c0 == c1);
        if (c0 != c1) {
            int *flag = reinterpret_cast<int *>(smem + G::OFF_FLAG);
            __threadfence();
            __syncthreads();
            if (tid == 0) *flag = atomicAdd(p.counters + c0, 1) == c1 - c0;
            __syncthreads();
            if (*flag) {                                                      // every piece is in the workspace
                __threadfence();
                if (tid == 0) p.counters[c0] = 0;
                attn_join<E, G::ROWS>(p.part, part_ml, c0, c1, rows, warp, lane, merged, D + G::PAD, ml);
                __syncthreads();
                finish(true);
            }
        }
        __syncthreads();                                                      // before the ring is filled again
        u += take;
    }
    if (pages_bad) atomicOr(error, pages_bad);
}

}  // namespace bqg
