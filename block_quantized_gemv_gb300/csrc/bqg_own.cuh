// bqg_own.cuh -- the second pass of attention behind shared prefixes: each sequence's own tokens.
//
// These are many short runs: 64 samples of one prompt with 8 KV heads are 512 (sequence, KV head) sets of a few hundred
// tokens.  attn_kernel gives a set's tokens to the four warps of a CTA in turns and then joins the warps, which costs 3
// to 4 us per piece, more than the tokens of a short set.  Here a piece is a warp's: the units of work are
// strips of 16 tokens in one line of all sets' (a set begins with kOwnLead that are no work), each warp takes a range
// of it, and nothing waits for another warp but the join of a set that several share.  Where there are fewer sets than
// warps each set begins with a range, so that no warp has two.
//
// A warp may begin while the first pass ends: only what it writes, and the first pass's rows, wait for that.  What it reads until then
// (lengths, tables, queries, the cache) a kernel before the call may have written.  That one is over: every kernel that may stand
// between waits before it signals, and this one begins when all CTAs of the last of them have signalled.  The fence keeps lines
// that this SM's L1 may hold from before out of it (up to 2 % of the call).  With a wait in its place 4 sequences behind 1000 tokens took 24 us
// instead of 16, 64 behind 8192 58 instead of 52.
//
// Measured (head_dim 128, as the pass alone, cold): 96 sequences of 75 to 300 tokens, 32 KV heads, q4_0: 41 us, attn_kernel 63, 12.4
// for the bytes; bound by issue (53 % of the slots, 580 instructions per strip of one row).  64 sequences of 125 to 500, 4 heads on each
// of 8, bf16: 30 us, attn_kernel 30, 12 for the bytes: 4 until the first strips are asked for, 11 of stream at the copy rate,
// 2 to 6 for the results, whose loads wait behind the stream's.
#pragma once

#include "bqg_attn.cuh"

namespace bqg {

// Strips of a range at least, and what beginning a set counts as.  The call's time (A: 96 sequences of 75 to 300 tokens behind 6 prefixes of
// 300, 32 KV heads, q4_0; B: 1024 x 50 behind 1000, 2 KV heads, bf16; C: 4 x 600 behind 1000, 8 KV heads, bf16):
//  * a lead of 0, 2, 4, 8: A 67, 64, 60, 61 us; B 80, 72, 67, 67;
//  * at least 4, 8, 16, 32: B 67, 67, 79, 95; C 21.7, 21.1, 24.0, 30.1; 4 x 77 behind 1000, q8_0: 18.2, 16.5, 16.4, 16.4.
constexpr int kOwnLeast = 8, kOwnLead = 4;

template <int FMT, int D, int RT> struct OwnGeom {
    using G = AttnGeom<FMT, D, RT>;
    static_assert(G::QREG, "queries in registers");
    static constexpr int ROWS = G::ROWS, S = G::S;
    // of a warp: the ring, whose memory holds the finished rows once it is drained; probabilities of the exact path;
    // new tokens that each row sees; softmax scales; biases
    static constexpr int MERGE = ROWS * (D + G::PAD) * 4;
    static constexpr int OFF_P = S * G::STAGE > MERGE ? S * G::STAGE : MERGE;
    static constexpr int OFF_VIS = OFF_P + 8 * kStrip * 4;
    static constexpr int OFF_RS = OFF_VIS + ROWS * 8;
    static constexpr int OFF_ML = OFF_RS + ROWS * 4;
    static constexpr int OFF_BIAS = OFF_ML + ROWS * 8;
    static constexpr int BYTES = (OFF_BIAS + (FMT == BQG_BF16 ? 0 : ROWS * G::NB * 4) + 127) / 128 * 128;
    static constexpr int SMEM = kAttnWarps * BYTES;
};

template <int FMT, int D, int RT>
__global__ void __launch_bounds__(32 * kAttnWarps) own_kernel(const SharedParams p, int *error)
{
    using G = AttnGeom<FMT, D, RT>;
    using O = OwnGeom<FMT, D, RT>;
    using A = AttnKernel<FMT, D, RT>;
    constexpr int S = G::S, MT = A::MT, ROWS = G::ROWS;
    constexpr float NEG = -__builtin_huge_valf();
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t *const own = smem + warp * O::BYTES;
    const uint32_t ring = smem_u32(own);
    float *const pw = reinterpret_cast<float *>(own + O::OFF_P);
    unsigned long long *const row_sees = reinterpret_cast<unsigned long long *>(own + O::OFF_VIS);
    float *const row_scale = reinterpret_cast<float *>(own + O::OFF_RS);
    float *const ml = reinterpret_cast<float *>(own + O::OFF_ML);
    float *const row_bias = reinterpret_cast<float *>(own + O::OFF_BIAS);
    float *const merged = reinterpret_cast<float *>(own);                     // [row][D + PAD]
    pdl_launch_dependents();
    __threadfence();                         // instead of a wait for the first pass: see above

    const int me = blockIdx.x * kAttnWarps + warp, workers = gridDim.x * kAttnWarps;
    auto strips_of = [&](const SharedSeq &q) { return (q.len + kStrip - 1) / kStrip - q.lo / kStrip; };
    int64_t per = 0;
    bool few = false;
    // a set's units: its strips and the lead, with few sets in whole ranges
    auto units_of = [&](const SharedSeq &q) {
        const int64_t n = strips_of(q) + kOwnLead;
        return few ? div_pos(n + per - 1, per) * per : n;
    };
    auto sets_of = [&](const SharedSeq &q) { return q.T ? (int64_t)p.cache.n_kv : 0; };
    auto weight = [&](const SharedSeq &q) { return sets_of(q) * units_of(q); };
    int bad = 0;
    int64_t mine, total;
    SharedSeq s;
    {
        int64_t sets = 0;
        total = attn_total(p, lane, [&](const SharedSeq &q) { sets += sets_of(q); return weight(q); }, bad, s, mine);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sets += __shfl_xor_sync(0xffffffffu, sets, o);
        // With few sets each begins with a range, so that a warp has one set's: at most total / per + sets ranges.  (Without it 4 x 77
        // behind 1000, q8_0, take 24 us instead of 16, 150 x 40 behind 300 37 instead of 31; nearer to as many sets as warps the
        // ranges that are left would be too long.)
        const bool fit = 8 * sets < 7 * (int64_t)workers;
        const int64_t to = fit ? workers - sets : workers;
        per = max(div_pos(total + to - 1, to), (int64_t)(kOwnLeast + kOwnLead));
        few = fit;
    }
    if (me == 0) {
        attn_check_ends(p, bad);
        if (bad) atomicOr(error, bad);
    }
    int64_t u = per * me, base = u;
    const int64_t u_end = few ? u + per : min(u + per, total);
    if (u < u_end) {
        mine = lane < p.n_seq ? weight(s) : 0;                                // (in whole ranges now)
        s = attn_find(p, u, lane, weight, s, mine, base);
    }
    if (u >= u_end || base > u) return pdl_wait();                            // (this launch does not end before the first pass's)
    int pages_bad = 0;

    while (u < u_end) {
        while (u - base >= weight(s)) {                                       // next sequence with work
            base += weight(s);
            s = attn_seq(p, s.b + 1, bad);
        }
        const int64_t off = u - base;
        const int strips = strips_of(s), rows = s.T * p.group;
        const int64_t all = units_of(s);
        const int h = (int)div_pos(off, all), first = (int)(off - (int64_t)h * all);
        const int take = (int)min((int64_t)(strips + kOwnLead - first), u_end - u);
        const int skip = max(first - kOwnLead, 0), n = first + take - kOwnLead - skip;     // strips of this piece
        if (n <= 0) {
            if (few) break;
            u += take;
            continue;
        }
        const int strip0 = skip + s.lo / kStrip;
        const int64_t seg0 = u - first + kOwnLead;                            // first strip of the whole set

        const int32_t *table = p.table + (int64_t)s.row * p.max_pages;
        // pages of strips j0 .. j0 + 31, one per lane
        auto pages_from = [&](int j0) {
            const int tok0 = (strip0 + j0 + lane) * kStrip;
            return j0 + lane < n ? table[tok0 >> p.cache.lp] : -1;
        };
        int pages = pages_from(0);
        QRegs<RT, G::KS> qf;
        typename A::RawQ raw[RT];
#pragma unroll
        for (int m = 0; m < RT; m++) A::fetch_q(p, s, h, 8 * m, lane, raw[m]);
        unsigned valid = 0;                                                   // stages whose page is in the cache
        auto issue = [&](int j, int st) {
            const int page = __shfl_sync(0xffffffffu, pages, j & 31);
            valid &= ~(1u << st);
            if (j < n) {
                const bool ok = page >= 0 && page < p.cache.n_pages;
                if (!ok) pages_bad = BQG_DEVERR_PAGE;
                valid |= (unsigned)ok << st;
                A::issue(p, s, h, (strip0 + j) * kStrip, page, ok, ring + st * G::STAGE, lane);
            }
            cp_async_commit();
            if ((j & 31) == 31) pages = pages_from(j + 1);
        };
#pragma unroll 1
        for (int j = 0; j < S - 1; j++) issue(j, j);
#pragma unroll
        for (int m = 0; m < RT; m++) {
            float scale, bias[G::NB];
            A::make_q(p, raw[m], qf.f[m], scale, bias);
            if (t == 0) {
                row_scale[8 * m + g] = scale;
                if constexpr (!A::BF)
#pragma unroll
                    for (int b = 0; b < G::NB; b++) row_bias[(m * G::NB + b) * 8 + g] = bias[b];
            }
        }
        if (lane < ROWS) row_sees[lane] = attn_sees(p, s, lane);
        __syncwarp();
        typename A::Rows r;
        r.begin(row_scale, t);
        int stage = 0;                                                        // j % S
#pragma unroll 1
        for (int j = 0; j < n; j++) {
            cp_async_wait<S - 2>();
            __syncwarp();
            issue(j + S - 1, stage ? stage - 1 : S - 1);
            const uint32_t st = ring + stage * G::STAGE;
            const bool ok = (valid >> stage) & 1;
            stage = stage + 1 == S ? 0 : stage + 1;
            const int tok0 = (strip0 + j) * kStrip;
            // the prefix's places in this sequence's page: whatever they hold, a NaN too, the result's bits are the same
            if (tok0 < s.lo) A::leave_out(st, s.lo - tok0, lane);
            A::strip(st, lane, qf, smem_u32(row_bias) + t * 8, row_sees, s, tok0, ok, pw, r);
        }
        cp_async_wait<0>();
        __syncwarp();                                                         // the ring's memory is free
#pragma unroll
        for (int m = 0; m < RT; m++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                r.sum[m][i] += __shfl_xor_sync(0xffffffffu, r.sum[m][i], 4);
                r.sum[m][i] += __shfl_xor_sync(0xffffffffu, r.sum[m][i], 8);
                r.sum[m][i] += __shfl_xor_sync(0xffffffffu, r.sum[m][i], 16);
                const int row = 8 * m + 2 * t + i;
                if (g == 0) {
                    ml[row * 2] = r.top[m][i];
                    ml[row * 2 + 1] = r.sum[m][i];
                }
                float *dst = merged + row * (D + G::PAD);
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
        __syncwarp();
        pdl_wait();                                                           // the first pass is over

        const int c0 = (int)div_pos(seg0, per), c1 = (int)div_pos(seg0 + strips - 1, per);   // warps that share the set
        constexpr int E = D / 32;                                             // values per lane of a row
        float *const part_ml = p.part + (int64_t)2 * workers * ROWS * D;
        bool last = c0 == c1;
        if (!last) {
            for (int row = 0; row < rows; row++) {
                const int64_t at = attn_slot_row<ROWS>(me, c0, row);
                float *dst = p.part + at * D + lane * E;
                const float *src = merged + row * (D + G::PAD) + lane * E;
#pragma unroll
                for (int e = 0; e < E; e += 2) *reinterpret_cast<float2 *>(dst + e) = *reinterpret_cast<const float2 *>(src + e);
                if (lane == 0) *reinterpret_cast<float2 *>(part_ml + at * 2) = make_float2(ml[row * 2], ml[row * 2 + 1]);
            }
            __threadfence();
            __syncwarp();
            int before = 0;
            if (lane == 0) before = atomicAdd(p.counters + c0, 1);
            last = __shfl_sync(0xffffffffu, before, 0) == c1 - c0;
            if (last) {                                                       // every piece is in the workspace
                __threadfence();
                if (lane == 0) p.counters[c0] = 0;
            }
        }
        if (last) {
            // the set's pieces in their order, and the prefix's row: loads of a few at a time
            constexpr int R = E <= 4 ? 4 : 2;
            for (int row = 0; row < rows; row += R) {
                float v[R][E], top[R], sum[R];
#pragma unroll
                for (int i = 0; i < R; i++) {
                    top[i] = NEG;
                    sum[i] = 0.f;
#pragma unroll
                    for (int e = 0; e < E; e++) v[i][e] = 0.f;
                }
                auto add = [&](int i, float m, float l, const float (&a)[E]) {
                    const float up = fmaxf(top[i], m);
                    const float old = up == top[i] ? 1.f : ex2(top[i] - up), now = up == m ? 1.f : ex2(m - up);
                    top[i] = up;
                    sum[i] = sum[i] * old + l * now;
#pragma unroll
                    for (int e = 0; e < E; e++) v[i][e] = v[i][e] * old + a[e] * now;
                };
                float2 q[R];
                float a[R][E];
                // (far: from four values to the next four)
                auto fetch = [&](int i, const float *m, const float *src, int far) {
                    q[i] = __ldcg(reinterpret_cast<const float2 *>(m));
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float2 f = __ldcg(reinterpret_cast<const float2 *>(src + e / 4 * far + e % 4));
                        a[i][e] = f.x; a[i][e + 1] = f.y;
                    }
                };
                for (int c = c0; c <= c1 && c0 != c1; c++) {
#pragma unroll
                    for (int i = 0; i < R; i++)
                        if (row + i < rows) {
                            const int64_t at = attn_slot_row<ROWS>(c, c0, row + i);
                            fetch(i, part_ml + at * 2, p.part + at * D + lane * E, 4);
                        }
#pragma unroll
                    for (int i = 0; i < R; i++)
                        if (row + i < rows) add(i, q[i].x, q[i].y, a[i]);
                }
                if (s.lo) {
#pragma unroll
                    for (int i = 0; i < R; i++)
                        if (row + i < rows) {
                            const int64_t at = shared_row(p, s, h, row + i);
                            fetch(i, p.rows_ml + at * 2, reinterpret_cast<const float *>(shared_at<D>(p, at, lane * E / 4)) + lane * E % 4, 128);
                        }
                }
                if (c0 == c1) {
#pragma unroll
                    for (int i = 0; i < R; i++)
                        if (row + i < rows) {
                            float f[E];
#pragma unroll
                            for (int e = 0; e < E; e++) f[e] = merged[(row + i) * (D + G::PAD) + lane * E + e];
                            add(i, ml[(row + i) * 2], ml[(row + i) * 2 + 1], f);
                        }
                }
#pragma unroll
                for (int i = 0; i < R; i++)
                    if (row + i < rows) {
                        if (s.lo) add(i, q[i].x, q[i].y, a[i]);
                        const int x = row + i, y = x / p.group;
                        attn_store_row<E>(p.out + ((int64_t)(s.q0 + y) * p.n_q + h * p.group + (x - y * p.group)) * D + lane * E, v[i], sum[i]);
                    }
            }
        }
        __syncwarp();                                                         // before the ring is filled again
        if (few) break;
        u += take;
    }
    pdl_wait();
    if (pages_bad) atomicOr(error, pages_bad);
}

}  // namespace bqg
