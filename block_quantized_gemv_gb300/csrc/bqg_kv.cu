// bqg_kv.cu -- per-head norm and rotation of queries and keys, the cache's
// encoder and decoder.
//
// norm_rope_kernel: a head row of one token is held by a warp, lane l the
// E = D / 32 values from E l on, so a row is one load of 4 to 32 bytes per lane,
// and a 32-value block sits in 32 / E neighbouring lanes.  A pair
// (i, i + R/2) is R/2/E lanes apart (R is a multiple of 16, E divides 8): one
// exchange; an adjacent pair is in one lane.  Everything is fp32 with the
// roundings of include/bqgemv.h; the sum of squares is kept as error-free fp32
// pairs, so r matches the fp64 definition up to a rare tie.
//
// It is a stream (bytes: rows in, queries out, cached rows out), but one row at a
// time per warp left it at 1.0 TB/s, bound by the instructions of the exact sum and
// their latency.  So a warp takes four rows of a token and one kind (queries, keys or
// values) together: their loads are in flight at once, and the next four's behind them; the
// arithmetic works on two rows per instruction (packed fp32, each half with
// its own rounding); the four sums are reduced together, each step halving the rows
// a lane still holds, and the reciprocal roots are taken once, each
// in the lanes that ended up with its row; the rotation's cos and sin are loaded once
// for the four rows.
//
// Measured (back to back): 7001 tokens of 64 + 8 + 8 heads of 128 values, bf16, norm and rotation: 97 us, bound by issue
// (about 150 instructions per row, 71 % of the slots); 8192 tokens of 8 + 8 heads, f32 into q4_0: 28 us, read back as bf16: 10.4 us,
// 0.6 of the copy rate; one token: 3.6 and 2.2 us, a launch's latency.
#include <algorithm>

#include "bqg_kv.cuh"

namespace bqg {

namespace {

constexpr int kWarps = 4;      // warps per CTA

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

// Two fp32 values, one per row, in one register pair: each operation rounds each of them once.
struct F2 { uint64_t v; };
__device__ __forceinline__ F2 f2(float a, float b) { F2 r; asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b)); return r; }
__device__ __forceinline__ float f2a(F2 x) { return __uint_as_float((uint32_t)x.v); }
__device__ __forceinline__ float f2b(F2 x) { return __uint_as_float((uint32_t)(x.v >> 32)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { F2 r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v)); return r; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { F2 r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v)); return r; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { F2 r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v)); return r; }
__device__ __forceinline__ F2 sub2(F2 a, F2 b) { return fma2(b, f2(-1.f, -1.f), a); }
// a + b where b may be a product: a packed product and the sum behind it would be
// fused into one rounding (measured: ptxas contracts mul.rn.f32x2 and add.rn.f32x2), so the
// sum is a 1 + b with a one that the compiler does not know.
__device__ __forceinline__ F2 add2_apart(F2 a, F2 b, F2 one) { return fma2(a, one, b); }
__device__ __forceinline__ void two_sum2(F2 a, F2 b, F2 &s, F2 &e, F2 one)
{
    s = add2_apart(a, b, one);
    const F2 bb = sub2(s, a);
    e = add2(sub2(a, sub2(s, bb)), sub2(b, bb));
}

// r = fp32(1 / sqrt(sum x^2 / D + eps)) of one row of the warp in fp64, for
// rows that leave the range of the pair arithmetic.
template <int E> __device__ __noinline__ float row_rms_recip_wide(const float (&x)[E], float eps)
{
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < E; i++) t = fma((double)x[i], (double)x[i], t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return (float)(1.0 / sqrt(t / (double)(E * 32) + (double)eps));
}

// r of the warp's four rows (x[pair][value]: rows 2 pair and 2 pair + 1), as pairs.
template <int E> __device__ __forceinline__ void rms_recip4(const F2 (&x)[2][E], bool f32, float eps, int lane, F2 one, F2 (&r)[2])
{
    F2 hi[2], lo[2];
#pragma unroll
    for (int p = 0; p < 2; p++) {
        hi[p] = mul2(x[p][0], x[p][0]);
        lo[p] = f32 ? fma2(x[p][0], x[p][0], mul2(hi[p], f2(-1.f, -1.f))) : f2(0.f, 0.f);   // the square's rounding (none: bf16)
#pragma unroll
        for (int i = 1; i < E; i++) {
            const F2 q = mul2(x[p][i], x[p][i]);
            F2 e;
            if (f32) lo[p] = add2(lo[p], fma2(x[p][i], x[p][i], mul2(q, f2(-1.f, -1.f))));
            two_sum2(hi[p], q, hi[p], e, one);
            lo[p] = add2(lo[p], e);
        }
    }
    // rows 0, 1 stay in lanes 0..15, rows 2, 3 in 16..31
    const bool up = lane & 16;
    auto xchg = [&](F2 v, int o) { F2 r; r.v = __shfl_xor_sync(0xffffffffu, (unsigned long long)v.v, o); return r; };
    F2 h = up ? hi[1] : hi[0], l = up ? lo[1] : lo[0], e;
    const F2 oh = xchg(up ? hi[0] : hi[1], 16), ol = xchg(up ? lo[0] : lo[1], 16);
    two_sum2(h, oh, h, e, one);
    l = add2(l, add2(ol, e));
    // the even row of the two in lanes with bit 3 clear, the odd one in the others
    const bool odd = lane & 8;
    SumSq t;
    t.hi = odd ? f2b(h) : f2a(h);
    t.lo = odd ? f2b(l) : f2a(l);
    t.merge(__shfl_xor_sync(0xffffffffu, odd ? f2a(h) : f2b(h), 8), __shfl_xor_sync(0xffffffffu, odd ? f2a(l) : f2b(l), 8));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t.merge(__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o));
    // (the eight lanes of a row differ at most in the order of their sums: the lowest one's counts)
    float mine = 0.f;
    const bool pair_ok = t.hi >= 0x1p-60f && t.hi <= 0x1p100f;
    if (pair_ok) mine = rms_recip_pair(t.hi, t.lo, (float)(E * 32), eps);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = __shfl_sync(0xffffffffu, mine, 8 * j);
    const unsigned bad = __ballot_sync(0xffffffffu, !pair_ok);
    if (bad & 0x01010101u) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if ((bad >> (8 * j)) & 1) {
                float row[E];
#pragma unroll
                for (int i = 0; i < E; i++) row[i] = (j & 1) ? f2b(x[j >> 1][i]) : f2a(x[j >> 1][i]);
                v[j] = row_rms_recip_wide<E>(row, eps);
            }
    }
    r[0] = f2(v[0], v[1]);
    r[1] = f2(v[2], v[3]);
}

// Larger of two magnitudes; a NaN stays.
__device__ __forceinline__ float max_abs_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// One row's codes as the format defines them, for what the quick path below leaves: lane's E values, d the
// scale of their block.
template <int FMT, int E> __device__ __noinline__ uint64_t codes_exact(const float (&y)[E], float d)
{
    uint64_t w = 0;
#pragma unroll
    for (int i = 0; i < E; i++) {
        uint32_t c;
        if constexpr (FMT == BQG_Q8_0) c = (uint32_t)q8_code(y[i], d) & 0xffu;
        else c = d != 0.0f ? (uint32_t)fminf(fmaxf(roundf(__fdiv_rn(y[i], d)) + 8.0f, 0.0f), 15.0f) : 8u;
        w |= (uint64_t)c << (8 * i);
    }
    return w;
}

// The warp's four rows (y[pair][value]: rows 2 pair and 2 pair + 1) into cache rows row, row + pitch, ...
//
// The four rows' block maxima are reduced together: each of the first two exchanges
// halves the rows a lane holds, so a row's scale is worked out in LB / 4 lanes of
// its block and handed to the others.  A code is round(x / d), halves away
// from zero, x / d rounded once to fp32.  The quick way is x times the approximate 1 / d, rounded by adding
// and taking off 1.5 x 2^23, two values per instruction.  It is off by at most 2^-22 of |x / d| (1 / d:
// 2^-23, the product and the quotient 2^-24 each), so by less than 2^-14 of a step for q8_0 (|x / d| up to 127.5) and 2^-18 for
// q4_0 (8.05); where a value lies within that of a half, or it or the scale is not an ordinary number, the
// rows' codes are divided out (one group of four rows in 16, and in 256; with 2^-12 for both it was one
// in four, and 8192 tokens of 8 heads took 39 us instead of 27).
template <int FMT, int D>
__device__ __forceinline__ void encode_rows(const F2 (&y)[2][D / 32], int rows, int lane, uint8_t *codes, uint16_t *scales,
                                            int64_t row, int64_t pitch)
{
    constexpr int E = D / 32, LB = 32 / E;            // lanes per block
    constexpr int RB = KvRow<FMT, D>::BYTES, NB = KvRow<FMT, D>::NB;
    auto value = [&](int j, int e) { return (j & 1) ? f2b(y[j >> 1][e]) : f2a(y[j >> 1][e]); };
    if constexpr (FMT == BQG_BF16) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            float one[E];
#pragma unroll
            for (int e = 0; e < E; e++) one[e] = value(j, e);
            if (j < rows) store_bf16<E>(reinterpret_cast<uint16_t *>(codes + (row + j * pitch) * RB) + lane * E, one);
        }
    } else {
        constexpr bool Q8 = (FMT == BQG_Q8_0);
        constexpr int S = Q8 ? 1 : 2;                 // largest magnitude; or largest value and largest negated value
        float a[4][S];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            a[j][0] = Q8 ? fabsf(value(j, 0)) : value(j, 0);
            if constexpr (!Q8) a[j][1] = -value(j, 0);
#pragma unroll
            for (int e = 1; e < E; e++) {
                a[j][0] = fmaxf(a[j][0], Q8 ? fabsf(value(j, e)) : value(j, e));
                if constexpr (!Q8) a[j][1] = fmaxf(a[j][1], -value(j, e));
            }
        }
        const bool up = lane & (LB / 2), up2 = lane & (LB / 4);
        float k[S];
#pragma unroll
        for (int i = 0; i < S; i++) {
            const float k0 = fmaxf(up ? a[2][i] : a[0][i], __shfl_xor_sync(0xffffffffu, up ? a[0][i] : a[2][i], LB / 2));
            const float k1 = fmaxf(up ? a[3][i] : a[1][i], __shfl_xor_sync(0xffffffffu, up ? a[1][i] : a[3][i], LB / 2));
            k[i] = fmaxf(up2 ? k1 : k0, __shfl_xor_sync(0xffffffffu, up2 ? k0 : k1, LB / 4));
#pragma unroll
            for (int o = LB / 8; o > 0; o >>= 1) k[i] = fmaxf(k[i], __shfl_xor_sync(0xffffffffu, k[i], o));
        }
        // this lane's row: 2 up + up2
        __half dh;
        bool odd;                                     // to be divided out
        if constexpr (Q8) {
            dh = __float2half_rn(__fdiv_rn(k[0], 127.0f));
        } else {
            dh = __float2half_rn(__fdiv_rn(k[0] > k[1] ? k[0] : -k[1], -8.0f));
        }
        float d = __half2float(dh), rd;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rd) : "f"(d));
        if constexpr (Q8) odd = !(k[0] * rd < 127.45f);
        else odd = k[0] == k[1] || !(fmaxf(k[0], k[1]) * fabsf(rd) < 8.05f);      // both signs of the largest: the first decides
        float near = odd ? 1.f : 0.f;
        uint32_t w[4][(E + 3) / 4];
        const float magic = Q8 ? 12582912.f : 12582920.f;                         // 1.5 x 2^23; q4_0: codes are round(x / d) + 8
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const int from = (lane & ~(LB - 1)) + p * (LB / 2);
            const F2 rd2 = f2(__shfl_sync(0xffffffffu, rd, from), __shfl_sync(0xffffffffu, rd, from + LB / 4));
            F2 m[E];
#pragma unroll
            for (int e = 0; e < E; e++) {
                F2 t = mul2(y[p][e], rd2);
                if constexpr (!Q8) t = f2(fminf(f2a(t), 7.0f), fminf(f2b(t), 7.0f));  // 15 is the last code (NaN: seen below)
                m[e] = add2(t, f2(magic, magic));
                const F2 f = sub2(mul2(y[p][e], rd2), sub2(m[e], f2(magic, magic)));
                const bool ca = !Q8 && f2a(t) == 7.0f, cb = !Q8 && f2b(t) == 7.0f;    // clipped: its own remainder says nothing
                near = max_abs_nan(near, ca && f2a(f) > 0.f ? 0.f : f2a(f));
                near = max_abs_nan(near, cb && f2b(f) > 0.f ? 0.f : f2b(f));
            }
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    auto bits = [&](int i) { return __float_as_uint(h ? f2b(m[i]) : f2a(m[i])); };
                    uint32_t u = __byte_perm(bits(e), bits(e + 1), 0x0040);
                    if constexpr (E >= 4) u = __byte_perm(u, __byte_perm(bits(e + 2), bits(e + 3), 0x0040), 0x5410);
                    w[2 * p + h][e / 4] = u;
                }
        }
        if (__any_sync(0xffffffffu, !(near < 0.5f - (Q8 ? 0x1p-14f : 0x1p-18f)))) {
            if constexpr (!Q8) {
                // the first value of largest magnitude of each row, in order
                float first = 0.f;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    float bv = value(j, 0), ba = fabsf(bv);
#pragma unroll
                    for (int e = 1; e < E; e++)
                        if (fabsf(value(j, e)) > ba) { bv = value(j, e); ba = fabsf(bv); }
                    int bl = lane;
#pragma unroll
                    for (int o = LB / 2; o > 0; o >>= 1) {
                        const float ov = __shfl_xor_sync(0xffffffffu, bv, o), oa = fabsf(ov);
                        const int ol = __shfl_xor_sync(0xffffffffu, bl, o);
                        if (oa > ba || (oa == ba && ol < bl)) { bv = ov; ba = oa; bl = ol; }
                    }
                    if (j == 2 * up + up2) first = bv;
                }
                dh = __float2half_rn(__fdiv_rn(first, -8.0f));
                d = __half2float(dh);
            }
            // The maxima pass over a NaN, and its code would be an ordinary one: a block that holds one has a NaN for its scale.
            // (q8_0 comes here 16 times as often as q4_0, which looks without asking: 8192 tokens of 8 heads 27.0 us with the
            // question and 27.9 without, q4_0 28.6 and 28.2.)
            if (!Q8 || __any_sync(0xffffffffu, isnan(near))) {
                bool nan = false;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    bool has = false;
#pragma unroll
                    for (int e = 0; e < E; e++) has |= isnan(value(j, e));
                    const unsigned lanes = __ballot_sync(0xffffffffu, has) >> (lane & ~(LB - 1));
                    if (j == 2 * up + up2) nan = lanes & ((1u << LB) - 1);
                }
                if (nan) {
                    dh = __ushort_as_half(0x7fff);
                    d = __half2float(dh);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float dj = __shfl_sync(0xffffffffu, d, (lane & ~(LB - 1)) + (j >> 1) * (LB / 2) + (j & 1) * (LB / 4));
                float one[E];
#pragma unroll
                for (int e = 0; e < E; e++) one[e] = value(j, e);
                const uint64_t c = codes_exact<FMT, E>(one, dj);
                w[j][0] = (uint32_t)c;
                if constexpr (E == 8) w[j][1] = (uint32_t)(c >> 32);
            }
        }
        // scales: by the first lane of those that worked a row's out
        const int mine = 2 * up + up2;
        if ((lane & (LB / 4 - 1)) == 0 && mine < rows) scales[(row + mine * pitch) * NB + lane / LB] = __half_as_ushort(dh);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            uint8_t *dst = codes + (row + j * pitch) * RB;
            if constexpr (!Q8) {
#pragma unroll
                for (int i = 0; i < (E + 3) / 4; i++) w[j][i] |= __shfl_xor_sync(0xffffffffu, w[j][i], LB / 2) << 4;   // the values 16 further on
            }
            if (j < rows && (Q8 || !up)) {
                uint8_t *at = Q8 ? dst + lane * E : dst + (lane / LB) * 16 + (lane % LB) * E;
                if constexpr (E == 2) *reinterpret_cast<uint16_t *>(at) = (uint16_t)w[j][0];
                else if constexpr (E == 4) *reinterpret_cast<uint32_t *>(at) = w[j][0];
                else *reinterpret_cast<uint2 *>(at) = make_uint2(w[j][0], w[j][1]);
            }
        }
    }
}

// CTAs per SM: registers allow so many, and a grid of that many has no second wave.  (D = 128, 7001 tokens: 95.8 us with six,
// 98.4 with seven, 104.3 with eight, whose registers spill.)
template <int D> constexpr int resident() { return D == 256 ? 3 : D == 128 ? 6 : 8; }

// Four rows of one token and kind, as loaded.
template <int E> struct RawRows { uint32_t w[4][E]; };       // fp32: E words a row; bf16: the first E / 2

template <int FMT, int D, bool F32> __global__ void __launch_bounds__(32 * kWarps, resident<D>()) norm_rope_kernel(const NormRopeParams p)
{
    constexpr int E = D / 32;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    // groups of four rows of a token: queries, then keys, then values
    const int gq = (p.n_q + 3) / 4, gk = p.k ? (p.n_kv + 3) / 4 : 0, gv = p.v ? (p.n_kv + 3) / 4 : 0, groups = gq + gk + gv;
    struct Item { int64_t t; int what, h, rows; };                            // what: 0 queries, 1 keys, 2 values
    auto item_of = [&](int64_t i) {
        Item m;
        m.t = (i >> 32) ? i / groups : (int64_t)((uint32_t)i / (uint32_t)groups);
        const int g = (int)(i - m.t * groups);
        m.what = g < gq ? 0 : g < gq + gk ? 1 : 2;
        m.h = 4 * (g - (m.what == 0 ? 0 : m.what == 1 ? gq : gq + gk));
        m.rows = min(4, (m.what ? p.n_kv : p.n_q) - m.h);
        return m;
    };
    auto load = [&](const Item &m, RawRows<E> &x) {
        const void *src = m.what == 0 ? p.q : m.what == 1 ? p.k : p.v;
        const int64_t first = m.t * (m.what == 0 ? p.q_stride : m.what == 1 ? p.k_stride : p.v_stride) + (int64_t)m.h * D + lane * E;
#pragma unroll
        for (int j = 0; j < 4; j++) {
#pragma unroll
            for (int i = 0; i < E; i++) x.w[j][i] = F32 ? 0x3f800000u : 0x3f803f80u;    // no row: ones, whose root is quick
            if (j < m.rows) {
                if constexpr (F32) {
                    const uint32_t *s = reinterpret_cast<const uint32_t *>(src) + first + j * D;
                    if constexpr (E == 2) {
                        const uint2 a = *reinterpret_cast<const uint2 *>(s);
                        x.w[j][0] = a.x; x.w[j][1] = a.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < E; i += 4) {
                            const uint4 a = *reinterpret_cast<const uint4 *>(s + i);
                            x.w[j][i] = a.x; x.w[j][i + 1] = a.y; x.w[j][i + 2] = a.z; x.w[j][i + 3] = a.w;
                        }
                    }
                } else {
                    const uint16_t *s = reinterpret_cast<const uint16_t *>(src) + first + j * D;
                    if constexpr (E == 2) {
                        x.w[j][0] = *reinterpret_cast<const uint32_t *>(s);
                    } else if constexpr (E == 4) {
                        const uint2 a = *reinterpret_cast<const uint2 *>(s);
                        x.w[j][0] = a.x; x.w[j][1] = a.y;
                    } else {
                        const uint4 a = *reinterpret_cast<const uint4 *>(s);
                        x.w[j][0] = a.x; x.w[j][1] = a.y; x.w[j][2] = a.z; x.w[j][3] = a.w;
                    }
                }
            }
        }
    };
    const float one_f = __int_as_float(0x3f800000 | (int)(p.T < 0));          // 1: the host lets no T < 0 through
    const F2 one = f2(one_f, one_f);
    const int64_t items = p.T * groups, step = (int64_t)gridDim.x * kWarps;
    int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i >= items) return;
    Item m = item_of(i);
    RawRows<E> raw;
    load(m, raw);
    for (;;) {
        // the position and slot of this token, the rows of the next item
        int64_t slot = -1;
        if (m.what && p.slots) slot = p.slots[m.t];
        int64_t pos = 0;
        const bool turn = m.what < 2 && p.rot;
        if (p.rot) pos = p.pos[m.t];
        F2 y[2][E];
#pragma unroll
        for (int a = 0; a < 2; a++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                if constexpr (F32) {
                    y[a][e] = f2(__uint_as_float(raw.w[2 * a][e]), __uint_as_float(raw.w[2 * a + 1][e]));
                } else {
                    const uint32_t u = raw.w[2 * a][e / 2], w = raw.w[2 * a + 1][e / 2];
                    y[a][e] = (e & 1) ? f2(bf16_hi(u), bf16_hi(w)) : f2(bf16_lo(u), bf16_lo(w));
                }
            }
        const Item now = m;
        const int64_t next = i + step;
        if (next < items) {
            m = item_of(next);
            load(m, raw);
        }

        // cos and sin of this lane's values (sin negated where the value is the first of its pair)
        float cs[E], sn[E];
        bool lost = false;
        const int half = p.rot / 2;
        const bool in = turn && lane * E < p.rot;
        int other = lane;
        if (turn) {
            lost = pos < 0 || pos >= p.n_pos;
            if (lost && lane == 0) atomicOr(p.error, BQG_DEVERR_POSITION);
            const float *row = p.table + (lost ? 0 : pos) * p.rot;
            if (in) {
                if (p.interleaved) {
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const int pair = (lane * E + e) / 2;
                        cs[e] = cs[e + 1] = row[pair];
                        sn[e + 1] = row[half + pair];
                        sn[e] = -sn[e + 1];
                    }
                } else {
                    const bool low = lane * E < half;
                    const int first = lane * E - (low ? 0 : half);
                    other = low ? lane + half / E : lane - half / E;
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float2 c = *reinterpret_cast<const float2 *>(row + first + e);
                        const float2 s = *reinterpret_cast<const float2 *>(row + half + first + e);
                        cs[e] = c.x; cs[e + 1] = c.y;
                        sn[e] = low ? -s.x : s.x; sn[e + 1] = low ? -s.y : s.y;
                    }
                }
            }
        }
        if (now.what < 2 && p.norm) {
            F2 r[2];
            rms_recip4<E>(y, F32, p.eps, lane, one, r);
            const float *g = now.what ? p.gamma_k : p.gamma_q;
            float gain[E];
            if (g) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 a = *reinterpret_cast<const float2 *>(g + lane * E + e);
                    gain[e] = a.x; gain[e + 1] = a.y;
                }
            }
#pragma unroll
            for (int a = 0; a < 2; a++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    y[a][e] = mul2(y[a][e], r[a]);
                    if (g) y[a][e] = mul2(y[a][e], f2(gain[e], gain[e]));
                }
        }
        if (turn) {
#pragma unroll
            for (int a = 0; a < 2; a++) {
                F2 o[E];                                                      // the pairs' other values
#pragma unroll
                for (int e = 0; e < E; e++) {
                    if (p.interleaved) o[e] = y[a][e ^ 1];
                    else o[e].v = __shfl_sync(0xffffffffu, (unsigned long long)y[a][e].v, other);
                }
                if (in) {
                    // a c - b s = a c + b (-s) and a s + b c: each product rounded, then their sum
#pragma unroll
                    for (int e = 0; e < E; e++)
                        y[a][e] = add2_apart(mul2(y[a][e], f2(cs[e], cs[e])), mul2(o[e], f2(sn[e], sn[e])), one);
                }
            }
        }
        if (slot >= 0 && !kv_slot_ok(p.cache, slot)) {
            if (lane == 0) atomicOr(p.error, BQG_DEVERR_SLOT);
            slot = -1;
        }
        if (now.what && p.slots) {
            // (a value is not turned, but without a position its token is not stored; its key's row reports it)
            if (!lost && slot >= 0 && (now.what < 2 || !p.rot || (pos >= 0 && pos < p.n_pos)))
                encode_rows<FMT, D>(y, now.rows, lane, now.what == 1 ? p.cache.k : p.cache.v,
                                    now.what == 1 ? p.cache.k_scale : p.cache.v_scale, kv_row(p.cache, slot, now.h),
                                    (int64_t)1 << p.cache.lp);
        } else {
            uint16_t *out = now.what ? p.k_out : p.q_out;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                float row[E];
#pragma unroll
                for (int e = 0; e < E; e++) row[e] = lost ? 0.f : (j & 1) ? f2b(y[j >> 1][e]) : f2a(y[j >> 1][e]);
                if (j < now.rows)
                    store_bf16<E>(out + (now.t * (now.what ? p.n_kv : p.n_q) + now.h + j) * D + lane * E, row);
            }
        }
        if (next >= items) break;
        i = next;
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
            atomicOr(p.error, BQG_DEVERR_SLOT);
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

template <int FMT, bool F32> void (*norm_rope_fn(int D))(NormRopeParams)
{
    return D == 64 ? norm_rope_kernel<FMT, 64, F32> : D == 128 ? norm_rope_kernel<FMT, 128, F32> : norm_rope_kernel<FMT, 256, F32>;
}
template <int FMT, bool F32> void (*kv_read_fn(int D))(KvReadParams)
{
    return D == 64 ? kv_read_kernel<FMT, 64, F32> : D == 128 ? kv_read_kernel<FMT, 128, F32> : kv_read_kernel<FMT, 256, F32>;
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int fmt, int D, int sms, cudaStream_t s, bool pdl)
{
    const int64_t groups = (p.n_q + 3) / 4 + ((p.k ? 1 : 0) + (p.v ? 1 : 0)) * ((p.n_kv + 3) / 4);
    const int64_t items = p.T * groups;
    if (items == 0) return cudaSuccess;
    if (cudaError_t e = device_error_word(&p.error)) return e;
    auto fn = p.x_f32 ? (fmt == BQG_Q8_0 ? norm_rope_fn<BQG_Q8_0, true>(D) : fmt == BQG_Q4_0 ? norm_rope_fn<BQG_Q4_0, true>(D) : norm_rope_fn<BQG_BF16, true>(D))
                      : (fmt == BQG_Q8_0 ? norm_rope_fn<BQG_Q8_0, false>(D) : fmt == BQG_Q4_0 ? norm_rope_fn<BQG_Q4_0, false>(D) : norm_rope_fn<BQG_BF16, false>(D));
    const int per_sm = D == 256 ? resident<256>() : D == 128 ? resident<128>() : resident<64>();
    return launch(fn, p, std::min<int64_t>((items + kWarps - 1) / kWarps, (int64_t)sms * per_sm), 32 * kWarps, s, pdl);
}

cudaError_t launch_kv_read(KvReadParams p, int fmt, int D, int out_f32, int sms, cudaStream_t s, bool pdl)
{
    const int64_t n = 2 * p.T * p.cache.n_kv * (D / 16);
    if (n == 0) return cudaSuccess;
    if (cudaError_t e = device_error_word(&p.error)) return e;
    auto fn = out_f32 ? (fmt == BQG_Q8_0 ? kv_read_fn<BQG_Q8_0, true>(D) : fmt == BQG_Q4_0 ? kv_read_fn<BQG_Q4_0, true>(D) : kv_read_fn<BQG_BF16, true>(D))
                      : (fmt == BQG_Q8_0 ? kv_read_fn<BQG_Q8_0, false>(D) : fmt == BQG_Q4_0 ? kv_read_fn<BQG_Q4_0, false>(D) : kv_read_fn<BQG_BF16, false>(D));
    return launch(fn, p, std::min<int64_t>((n + 255) / 256, (int64_t)sms * 8), 256, s, pdl);
}

}  // namespace bqg
