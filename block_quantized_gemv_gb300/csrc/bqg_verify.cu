// bqg_verify.cu -- drafted tokens against the target's probabilities.
//
// With p the target's distribution after a token and q the draft's, a token's drafts are taken in their order: t is
// accepted when u q(t) Z < r(t), r = p and Z = 1 before the first rejection; a rejection makes
//     r(x) = max(p(x) - c q(x), 0),  c the sum of the Z so far,  Z = sum of the new r,
// (taking off Z q from what is left each time comes to c q from p, since q >= 0, so nothing is stored), and the next
// token is the first one at which the running sum of r exceeds u' times the whole.  Chosen drafts have q = 1 at their
// token: r is p without the rejected tokens, Z = 1 - their p, and no sum is needed but the last.
//
//  * What decides on the drafts is a handful of numbers, loaded at once; a row of p (and q) is only read where a
//    sum is needed: once per rejection of a sampled draft, once for the next token (the last rejection's sum serves for
//    it).  So it is a stream of one or two rows per sequence, and for few sequences latency.
//  * A cluster of up to 8 CTAs takes a sequence, each warp a contiguous part of the row.  The first warp walks the tree and
//    puts its orders (a sum, or the end) into every CTA's shared memory, two cluster barriers for each: who arrives how
//    often is decided in one place.
//  * An answer is a whole number and depends on where a sum of up to 2^18 terms crosses a border, so fp32 sums (off by 1e-7:
//    another token once in some hundred draws) would not do, and fp64's rate is 1/64 of fp32's here: p - c q is
//    formed as an fp32 pair, off by 2^-47 of what c takes off beyond the first rejection (rest2), and added with error-free sums, two
//    at a time: about 2^-45 of the sum, or of the largest one behind that token, the first rejection's.  The walk's few numbers are pairs too: with fp64 a draft cost 900 cycles, with pairs 200.
//  * The crossing is looked for in the warps' sums, then by the warp that holds it in the sums that it kept (of 32 lanes and up
//    to 16 steps), then in the 16 bytes of one lane: nothing of the row is read again but those.  There the sums are
//    whole numbers of 2^-61 of all.  (Reading the warp's part again took 7 us of 18, most of it for fetching instructions that run once.)
//  * Measured: one chain of 5 sampled drafts, 32,000 tokens, fp32: 9.4 us: about 3 for the launch, 1.6 until the deciding numbers
//    are there, 3 for the rejection's sum (barriers 1.2), 1.9 for the token.  16 chosen trees, 100,003, bf16: 12 us.  64 sampled trees
//    of up to 10, 131,072, fp32: 44 us, 10 for the bytes: the first sums run at the copy rate; then trees with up to five rejections wait
//    for one pass after the other, from L2 (2.5 to 7 us each).
#include <climits>

#include <cooperative_groups.h>

#include "bqg_verify.cuh"

namespace bqg {

namespace {

constexpr int kMaxCtas = 8, kMaxDrafts = 64;
// Values of a row that a CTA is taken for.  With 512, 2048, 8192, 32768 (trees of 6): 1 sequence of 1000, fp32: 8.9, 7.2, 7.2, 7.2 us; of
// 5000: 9.3, 9.0, 8.5, 8.5; of 32,000: 9.4, 9.4, 10.0, 15.5; 64 of 32,000: 25, 25, 34, 53; 128 of 5000, bf16: 15.8, 9.6, 8.8, 8.8.
constexpr int kLeast = 2048;

// An unevaluated sum of two fp32 numbers, none of which is negative.
struct Pair {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float h, float l)
    {
        // the smaller number's error in the sum is exact (Dekker): five operations, two_sum takes six
        const float a = fmaxf(hi, h), b = fminf(hi, h);
        hi = __fadd_rn(a, b);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(b, __fsub_rn(hi, a)), l));
    }
    // the same sum, hi the nearest fp32 number to it (|hi| >= |lo|): what is added to lo afterwards is rounded to 2^-48 of hi, where
    // the errors of n additions that lo had gathered would make that n 2^-48
    __device__ __forceinline__ void tidy()
    {
        const float s = __fadd_rn(hi, lo);
        lo = __fsub_rn(lo, __fsub_rn(s, hi));
        hi = s;
    }
};
// hi + lo of a pair, hi the nearest fp32 number (|hi| >= |lo| or near it).
__device__ __forceinline__ Pair tidy(float hi, float lo)
{
    Pair r;
    two_sum(hi, lo, r.hi, r.lo);
    return r;
}
// An unevaluated sum of three, for what large numbers that are all but equal are taken off from each other with: a pair would know
// the small rest of them to 2^-48 of the large ones.
struct Triple {
    float hi = 0.f, mid = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        float h, m, e;
        two_sum(hi, x, h, e);
        two_sum(mid, e, m, e);
        lo = __fadd_rn(lo, e);
        two_sum(h, m, hi, m);
        two_sum(m, lo, mid, lo);
    }
};
// Parts of a row's sum as whole numbers: units of about 2^-61 of it, so that what follows is exact and quick (fp64 takes
// 16 cycles per warp and operation here, and its latency).
struct Units {
    float by[2];                       // two powers of two: one would leave fp32's range for sums below 2^-66
    __device__ __forceinline__ explicit Units(float whole)
    {
        const int k = 60 - (int)(__float_as_uint(whole) >> 23) + 127;             // (a denormal one counts as 2^-127)
        const int a = k >> 1, b = k - a;
        by[0] = __uint_as_float((uint32_t)(127 + a) << 23);
        by[1] = __uint_as_float((uint32_t)(127 + b) << 23);
    }
    __device__ __forceinline__ long long of(float x) const { return __float2ll_rn(__fmul_rn(__fmul_rn(x, by[0]), by[1])); }
    // (what is less than a unit still counts as something)
    __device__ __forceinline__ long long of(const Pair &v) const { return max(of(v.hi) + of(v.lo), (long long)(__fadd_rn(v.hi, v.lo) > 0.f)); }
};

// Two numbers per register pair, each rounded by itself.
struct F2 { uint64_t v; };
__device__ __forceinline__ F2 f2(float a, float b) { F2 r; asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b)); return r; }
__device__ __forceinline__ float lower(F2 x) { return __uint_as_float((uint32_t)x.v); }
__device__ __forceinline__ float upper(F2 x) { return __uint_as_float((uint32_t)(x.v >> 32)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { F2 r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v)); return r; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { F2 r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v)); return r; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { F2 r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v)); return r; }
__device__ __forceinline__ F2 sub2(F2 a, F2 b) { return fma2(b, f2(-1.f, -1.f), a); }      // (one rounding: b times -1 is exact)
// Two pairs at once.
struct Pair2 {
    F2 hi, lo;
    __device__ __forceinline__ void add(F2 h, F2 l)
    {
        const F2 s = add2(hi, h), b = sub2(s, hi);
        const F2 e = add2(sub2(hi, sub2(s, b)), sub2(h, b));       // Knuth's: no comparison, which would not be packed
        hi = s;
        lo = add2(lo, add2(e, l));
    }
    __device__ __forceinline__ void tidy()
    {
        const F2 s = add2(hi, lo);
        lo = sub2(lo, sub2(s, hi));
        hi = s;
    }
    __device__ __forceinline__ Pair both() const
    {
        Pair r{lower(hi), lower(lo)};
        r.add(upper(hi), upper(lo));
        return r;
    }
};

struct Order {
    int sum;                           // 0: the end; the token is looked for with what follows as it was
    int row;                           // of target and draft
    int minus;                         // 1: r is max(p - (1 + s) q, 0); 0: p (and s is 0)
    Pair s;
    int at;                            // the end: which of all warps looks for the token (-1: none does)
    float whole;                       // ... with Units(whole)
    long long goal;
    int n_gone;                        // chosen drafts that were rejected here
    int gone[kMaxDrafts];
};

// A probability: from 0 to 1 (a NaN: 0).
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }
template <bool F32> __device__ __forceinline__ float load_raw(const void *x, int64_t i)
{
    if constexpr (F32) return __ldg(reinterpret_cast<const float *>(x) + i);
    else return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(x) + i) << 16);
}
template <bool F32> __device__ __forceinline__ float load_prob(const void *x, int64_t i) { return prob(load_raw<F32>(x, i)); }
// One row: probabilities of `vocab` tokens, of which 16 bytes are loaded at once where they lie on such a boundary and in the row.
template <bool F32> struct Row {
    static constexpr int E = F32 ? 4 : 8;                  // values of 16 bytes
    const uint8_t *at;
    int vocab, off;                                        // off: tokens x with (x + off) % E == 0 lie on a boundary
    __device__ __forceinline__ Row(const void *base, int64_t first, int vocab)
        : at(reinterpret_cast<const uint8_t *>(base) + first * (F32 ? 4 : 2)), vocab(vocab),
          off((int)(reinterpret_cast<uintptr_t>(at) / (F32 ? 4 : 2)) & (E - 1))
    {
    }
    // tokens x .. x + E - 1 as they lie, zeros where they are none; `there`: they lie on a boundary
    __device__ __forceinline__ uint4 load(int x, bool there) const
    {
        if (there && x >= 0 && x <= vocab - E) return __ldg(reinterpret_cast<const uint4 *>(at + (int64_t)x * (F32 ? 4 : 2)));
        return one_by_one(at, x, vocab);
    }
    static __device__ __noinline__ uint4 one_by_one(const uint8_t *at, int x, int vocab)
    {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < E; i++)
            if (x + i >= 0 && x + i < vocab) {
                if constexpr (F32) w[i % 4] = __ldg(reinterpret_cast<const uint32_t *>(at) + x + i);
                else w[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(at) + x + i) << (16 * (i & 1));
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void values(const uint4 &q, float (&v)[E])
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < E; i++) v[i] = prob(F32 ? __uint_as_float(w[i % 4]) : (i & 1) ? bf16_hi(w[i / 2 % 4]) : bf16_lo(w[i / 2 % 4]));
    }
};

// max(p - c q, 0) of two tokens, as pairs, with c = 1 + s; ONE: s is 0, as it is after a first rejection.
// p and c q may be all but equal over a whole row (a draft near its target), and what is left of them decides.  So it is
// formed as (p - q) - s q, the first difference exact, the product's error along with it, the sign taken from all of it: off by
// 2^-47 of s q and of itself, where a rounded c q or c would be off by as much of c q.
template <bool ONE> __device__ __forceinline__ void rest2(float p0, float p1, float q0, float q1, const Pair &s, F2 &hi, F2 &lo)
{
    const F2 a = f2(fmaxf(p0, q0), fmaxf(p1, q1)), q = f2(q0, q1);
    hi = sub2(a, q);                                               // a - q and its error, exact as a >= q
    lo = sub2(sub2(a, hi), q);
    if constexpr (!ONE) {
        const F2 m = mul2(q, f2(s.hi, s.hi));
        const F2 e = fma2(q, f2(-s.lo, -s.lo), fma2(q, f2(-s.hi, -s.hi), m));      // m - s q
        const F2 h = sub2(hi, m);                                  // as above where something is left
        lo = add2(sub2(sub2(hi, h), m), add2(lo, e));
        const F2 all = add2(h, lo);
        hi = f2(lower(all) > 0.f ? lower(h) : 0.f, upper(all) > 0.f ? upper(h) : 0.f);
        lo = f2(lower(all) > 0.f ? lower(lo) : 0.f, upper(all) > 0.f ? upper(lo) : 0.f);
    }
}
// Of one.
__device__ __forceinline__ Pair rest(float p, float q, const Pair &s)
{
    F2 hi, lo;
    rest2<false>(p, p, q, q, s, hi, lo);
    return Pair{lower(hi), lower(lo)};
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

template <bool F32, bool DRAFT, int kWarps> struct Verify {
    static constexpr int E = Row<F32>::E;
    static constexpr int kStep = 32 * E;                  // values that a warp takes at once: 16 bytes per lane
    static constexpr int kKept = kWarps == 16 ? 8 : 16;   // parts of a warp's range whose sums are kept
    static constexpr int U = kWarps == 16 && !DRAFT ? 4 : 2;   // steps whose loads are in flight together

    // Which of the rejected tokens lie in [a, e).
    static __device__ __forceinline__ unsigned long long gone_in(const Order &o, int a, int e, int lane)
    {
        if (DRAFT) return 0;
        const bool lo = lane < o.n_gone && o.gone[lane] >= a && o.gone[lane] < e;
        const bool hi = lane + 32 < o.n_gone && o.gone[lane + 32] >= a && o.gone[lane + 32] < e;
        return (unsigned long long)__ballot_sync(0xffffffffu, lo) | (unsigned long long)__ballot_sync(0xffffffffu, hi) << 32;
    }
    // The sum of r over the E tokens from x on.
    template <bool FIRST>
    static __device__ __forceinline__ Pair2 some(const Order &o, const uint4 &pw, const uint4 &qw, int x, unsigned long long gone)
    {
        float p[E], q[E];
        Row<F32>::values(pw, p);
        if constexpr (DRAFT) Row<F32>::values(qw, q);
        if (!DRAFT && gone) {
#pragma unroll 1
            for (unsigned long long g = gone; g; g &= g - 1) {
                const int at = o.gone[__ffsll(g) - 1] - x;
#pragma unroll
                for (int i = 0; i < E; i++)
                    if (at == i) p[i] = 0.f;
            }
        }
        Pair2 s;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            F2 hi = f2(p[i], p[i + 1]), lo = f2(0.f, 0.f);
            if constexpr (DRAFT) rest2<FIRST>(p[i], p[i + 1], q[i], q[i + 1], o.s, hi, lo);
            if (i == 0) { s.hi = hi; s.lo = lo; }
            else s.add(hi, lo);
        }
        return s;
    }
    // The sum of r over a warp's tokens, from a on and before e, in lane 0.  kept[k][lane]: the sums of the lane's tokens in the k-th
    // `steps` steps of it, its part k.
    template <bool FIRST>
    static __device__ __forceinline__ Pair sum(const VerifyParams &p, const Order &o, int a, int e, int steps, float2 (*kept)[32], int lane)
    {
        const Row<F32> target(p.target, (int64_t)o.row * p.target_stride, p.vocab), draft(p.draft, (int64_t)o.row * p.draft_stride, p.vocab);
        const unsigned long long gone = gone_in(o, a, e, lane);
        const bool q = DRAFT && o.minus;
        Pair all;
        Pair2 part{f2(0.f, 0.f), f2(0.f, 0.f)};
        int left = steps;                                              // of the part
#pragma unroll 1
        for (int k0 = 0; a + k0 * kStep < e; k0 += U) {
            uint4 pw[U], qw[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int x = a + (k0 + u) * kStep + E * lane;
                pw[u] = qw[u] = make_uint4(0, 0, 0, 0);
                if (x < e) {
                    pw[u] = target.load(x, true);
                    if (q) qw[u] = draft.load(x, draft.off == target.off);
                }
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int x = a + (k0 + u) * kStep;
                if (x >= e) break;
                const Pair2 s = some<FIRST>(o, pw[u], qw[u], x + E * lane, gone);
                if (left == steps) {
                    part = s;
                } else {
                    part.add(s.hi, s.lo);
                    part.tidy();
                }
                if (--left == 0 || x + kStep >= e) {
                    const Pair one = part.both();
                    (*kept++)[lane] = make_float2(one.hi, one.lo);
                    all.add(one.hi, one.lo);
                    all.tidy();
                    left = steps;
                }
            }
        }
        return over_lanes(all);
    }
    static __device__ __forceinline__ Pair over_lanes(Pair v)
    {
#pragma unroll 1
        for (int s = 16; s > 0; s >>= 1) v.add(__shfl_xor_sync(0xffffffffu, v.hi, s), __shfl_xor_sync(0xffffffffu, v.lo, s));
        return v;
    }
    // The first of 32 consecutive parts (this lane's: v) whose running sum exceeds `goal`, which then is what is left of the
    // goal in that part.  Without one, which is a matter of rounding, the last part that is not nothing, and the goal is out of reach.
    static __device__ __noinline__ int cross(long long v, long long &goal, int lane)
    {
        long long run = v;
#pragma unroll 1
        for (int s = 1; s < 32; s <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, run, s);
            if (lane >= s) run += o;
        }
        const unsigned some = __ballot_sync(0xffffffffu, v > 0), past = __ballot_sync(0xffffffffu, run > goal) & some;
        const int at = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
        goal = past ? goal - __shfl_sync(0xffffffffu, run - v, at) : LLONG_MAX;
        return at;
    }
    static __device__ __forceinline__ long long over_lanes(long long v)
    {
#pragma unroll 1
        for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
        return v;
    }
    // ... among a warp's tokens, from a on and before e, whose sums are kept.
    static __device__ __forceinline__ int token(const VerifyParams &p, const Order &o, int a, int e, int steps, const float2 (*kept)[32],
                                                const Units &units, long long goal, int lane)
    {
        // the kept part: 32 / kKept lanes add up one (from different banks)
        constexpr int L = 32 / kKept;
        Pair s;
        const int k = lane / L;
        if (a + k * steps * kStep < e) {
#pragma unroll 4
            for (int i = 0; i < 32 / L; i++) {
                const float2 f = kept[k][lane % L * (32 / L) + ((i + k) & (32 / L - 1))];
                s.add(f.x, f.y);
            }
        }
#pragma unroll
        for (int i = 1; i < L; i <<= 1) s.add(__shfl_xor_sync(0xffffffffu, s.hi, i), __shfl_xor_sync(0xffffffffu, s.lo, i));
        const int part = cross(lane % L ? 0 : units.of(s), goal, lane) / L;
        a += part * steps * kStep;
        const Row<F32> target(p.target, (int64_t)o.row * p.target_stride, p.vocab), draft(p.draft, (int64_t)o.row * p.draft_stride, p.vocab);
        const bool q = DRAFT && o.minus;
        long long v;
        if (steps == 1) {
            const float2 f = kept[part][lane];
            v = units.of(Pair{f.x, f.y});
        } else {
            v = step_of(o, target, draft, a, min(a + steps * kStep, e), units, goal, lane);
        }
        // the lane, then its token
        const int l = cross(v, goal, lane), x = a + E * l + lane;
        Pair r{0.f, 0.f};
        if (lane < E && x >= 0 && x < e) {
            r.hi = load_prob<F32>(target.at, x);
            if constexpr (DRAFT)
                if (q) r = rest(r.hi, load_prob<F32>(draft.at, x), o.s);
            if (!DRAFT)
                for (int i = 0; i < o.n_gone; i++)
                    if (o.gone[i] == x) r.hi = 0.f;
        }
        return a + E * l + cross(units.of(r), goal, lane);
    }
    // The step of a part of several, as `a`; returns this lane's share of it.
    static __device__ __noinline__ long long step_of(const Order &o, const Row<F32> &target, const Row<F32> &draft, int &a, int e,
                                                     const Units &units, long long &goal, int lane)
    {
        const unsigned long long gone = gone_in(o, a, e, lane);
        const int first = a;
        int last = -1;
#pragma unroll 1
        for (;;) {
            const int x = a + E * lane;
            uint4 pw = make_uint4(0, 0, 0, 0), qw = pw;
            if (x < e) {
                pw = target.load(x, true);
                if (DRAFT && o.minus) qw = draft.load(x, draft.off == target.off);
            }
            const long long v = units.of(some<false>(o, pw, qw, x, gone).both()), all = over_lanes(v);
            if (all > goal || last == a) return v;
            if (all > 0) last = a;
            if (goal != LLONG_MAX) goal -= all;
            a += kStep;
            if (a >= e) {                                              // rounding: the last one that is not nothing
                goal = LLONG_MAX;
                a = last = last < 0 ? first : last;
            }
        }
    }
};

// A draft as the walk needs it.
struct Draft {
    float u, p, q;
    int token;
};
// u q Z < r(t) of it, r as a pair.
__device__ __forceinline__ bool accepted(const Draft &d, const Pair &r, const Pair &Z)
{
    const float m = __fmul_rn(d.u, d.q), me = fmaf(d.u, d.q, -m);
    const float y = __fmul_rn(m, Z.hi), ye = __fadd_rn(fmaf(m, Z.hi, -y), fmaf(m, Z.lo, __fmul_rn(me, Z.hi)));
    // near each other their difference is exact
    return __fadd_rn(__fsub_rn(y, r.hi), __fsub_rn(ye, r.lo)) < 0.f;
}

template <bool F32, bool DRAFT, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 8 ? 4 : 2) verify_kernel(const VerifyParams p, int ctas)
{
    namespace cg = cooperative_groups;
    using V = Verify<F32, DRAFT, kWarps>;
    __shared__ Order order;
    __shared__ Pair warp_sum[kWarps];
    __shared__ float2 kept[kWarps][V::kKept][32];
    __shared__ Draft drafts[kMaxDrafts];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % ctas, b = blockIdx.x / ctas;
    const bool walker = rank == 0 && warp == 0;
    pdl_wait();
    pdl_launch_dependents();

    // A warp's part of a row: whole steps from a boundary of 16 bytes on, which for the first one is up to E - 1 values before the row.
    int steps;                                 // of a kept part
    auto range = [&](int row, int w, int &a, int &e) {
        const int off = Row<F32>(p.target, (int64_t)row * p.target_stride, p.vocab).off;
        const int all = (p.vocab + off + V::kStep - 1) / V::kStep, per = (all + ctas * kWarps - 1) / (ctas * kWarps);
        steps = (per + V::kKept - 1) / V::kKept;
        a = min(w * per, all) * V::kStep - off;
        e = min(a + per * V::kStep, p.vocab);
    };
    auto meet = [&]() {
        if (ctas == 1) return __syncthreads();
        cluster_arrive();
        cluster_wait();
    };
    // One round: the order is in every CTA's shared memory, then the CTAs' sums are in theirs.  (After the end's order
    // nobody reads another CTA's memory.)
    auto round = [&]() {
        meet();
        if (!order.sum) {
            if (order.at == rank * kWarps + warp) {
                int a, e;
                range(order.row, order.at, a, e);
                const int x = V::token(p, order, a, e, steps, kept[warp], Units(order.whole), order.goal, lane);
                if (lane == 0) p.next_token[b] = min(max(x, 0), p.vocab - 1);
            }
            return false;
        }
        int a, e;
        range(order.row, rank * kWarps + warp, a, e);
        const Pair s = order.s.hi == 0.f && order.s.lo == 0.f ? V::template sum<true>(p, order, a, e, steps, kept[warp], lane)
                                                              : V::template sum<false>(p, order, a, e, steps, kept[warp], lane);
        if (lane == 0) warp_sum[warp] = s;
        meet();
        return true;
    };
    if (ctas > 1) cluster_arrive();            // every CTA has begun, before others write to its shared memory
    if (!walker) {
        if (ctas > 1) cluster_wait();
        while (round()) {}
        return;
    }

    // ---------------- the first CTA's first warp walks ----------------
    const int64_t a0 = p.q_start[b], e0 = p.q_start[b + 1];
    const int64_t q0 = min(max(a0, (int64_t)0), p.n_tokens), q1 = min(max(e0, q0), p.n_tokens);
    const int T = (int)min(q1 - q0, (int64_t)p.max_q);
    int bad = q0 != a0 || q1 != e0 || T != q1 - q0 ? BQG_DEVERR_LENGTH : 0;
    if (b == 0 && (a0 != 0 || p.q_start[p.n_seq] != p.n_tokens)) bad |= BQG_DEVERR_LENGTH;
    // drafts `lane` and 32 on
    int up[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int i = lane + 32 * j;
        up[j] = -1;
        if (i >= T) continue;
        Draft d{p.u[q0 + i], 0.f, 1.f, -1};
        if (i) {
            d.token = p.tokens[q0 + i];
            up[j] = p.parent ? p.parent[q0 + i] : i - 1;
            if (up[j] < 0 || up[j] >= i || d.token < 0 || d.token >= p.vocab) {
                bad |= BQG_DEVERR_DRAFT;
                up[j] = -1;
            } else {
                const int64_t row = q0 + up[j];
                d.p = load_prob<F32>(p.target, row * p.target_stride + d.token);
                if constexpr (DRAFT) d.q = load_prob<F32>(p.draft, row * p.draft_stride + d.token);
            }
        }
        drafts[i] = d;
    }
    if (bad) atomicOr(p.error, bad);
    __syncwarp();
    if (ctas > 1) cluster_wait();
    const Pair one{1.f, 0.f};
    // A round: the warps' sums, in their order, each lane the next few.
    constexpr int NE = kMaxCtas * kWarps / 32;
    const int each = max(ctas * kWarps / 32, 1);
    Pair parts[NE];
    auto give = [&](int sum, int64_t row, const Pair &s, int minus, int n_gone, int at = -1, float whole = 1.f, long long goal = 0) {
        __syncwarp();
        if (lane < ctas) {                                // to one CTA per lane
            Order *o = ctas > 1 ? cluster.map_shared_rank(&order, lane) : &order;
            o->sum = sum;
            o->at = at;
            o->whole = whole;
            o->goal = goal;
            if (sum) {
                o->row = (int)row;
                o->s = s;
                o->minus = minus;
                o->n_gone = n_gone;
                if (lane)
                    for (int i = 0; i < n_gone; i++) o->gone[i] = order.gone[i];
            }
        }
        __syncwarp();
        if (!round()) return Pair();
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const int w = lane * each + i;
            parts[i] = Pair();
            if (i < each && w < ctas * kWarps)
                parts[i] = ctas > 1 ? *cluster.map_shared_rank(&warp_sum[w % kWarps], w / kWarps) : warp_sum[w];
        }
        Pair z;
#pragma unroll
        for (int i = 0; i < NE; i++) z.add(parts[i].hi, parts[i].lo);
        z = V::over_lanes(z);
        return tidy(__shfl_sync(0xffffffffu, z.hi, 0), __shfl_sync(0xffffffffu, z.lo, 0));
    };
    int node = 0, count = T > 0, place[2] = {lane == 0 && T > 0 ? 0 : -1, -1};   // place: of the path
    int finder = -1;                                      // the warp that holds the next token
    float whole = 1.f;
    long long goal = 0;
    if (T > 0) {
        int last = 0, n_gone = 0;                         // the last draft looked at
        Pair Z = one, s;                                  // c = minus + s
        int minus = 0;
        Triple left{1.f, 0.f, 0.f};                       // chosen drafts: Z
        bool known = false;                               // `parts` and what the CTAs hold are those of r
        for (;;) {
            unsigned long long below = (unsigned long long)__ballot_sync(0xffffffffu, up[0] == node) |
                                       (unsigned long long)__ballot_sync(0xffffffffu, up[1] == node) << 32;
            below &= last < 63 ? ~0ull << (last + 1) : 0ull;
            if (!below) break;
            const int i = __ffsll(below) - 1;
            last = i;
            Draft d = drafts[i];
            Pair r{d.p, 0.f};
            if constexpr (DRAFT) {
                r = rest(d.p, minus ? d.q : 0.f, s);
            } else {
                const bool again = (lane < n_gone && order.gone[lane] == d.token) || (lane + 32 < n_gone && order.gone[lane + 32] == d.token);
                if (__any_sync(0xffffffffu, again)) r.hi = 0.f;
            }
            if (accepted(d, r, Z)) {
                node = i;
                if (lane == (count & 31)) place[count >> 5] = i;
                count++;
                Z = one;
                minus = 0;
                s = Pair();
                left = Triple{1.f, 0.f, 0.f};
                n_gone = 0;
                known = false;
            } else if constexpr (DRAFT) {
                if (minus) {
                    s.add(Z.hi, Z.lo);
                    s.tidy();
                }
                minus = 1;
                Z = give(1, q0 + node, s, minus, 0);
                known = true;
            } else {
                left.add(-r.hi);
                Z = Pair{left.hi, left.mid};
                __syncwarp();
                if (lane == 0) order.gone[n_gone] = d.token;
                n_gone++;
                __syncwarp();
            }
        }
        if (!known) {
            Z = give(1, q0 + node, Pair(), 0, n_gone);
        }
        if (!(Z.hi > 0.f) && (known || n_gone)) {         // nothing left: the target's own
            Z = give(1, q0 + node, Pair(), 0, 0);
        }
        if (Z.hi > 0.f) {
            // u Z: what the running sum has to exceed, in whole units
            whole = Z.hi;
            const Units units(whole);
            const float u = drafts[0].u;
            const float m = __fmul_rn(u, Z.hi), me = fmaf(u, Z.hi, -m);
            goal = (u >= 0.f ? units.of(m) : 0) + __float2ll_rd(__fmul_rn(__fmul_rn(fmaf(u, Z.lo, me), units.by[0]), units.by[1]));
            // the lane's warps, then the warp
            long long part[NE], sum = 0;
#pragma unroll
            for (int i = 0; i < NE; i++) {
                part[i] = units.of(parts[i]);
                sum += part[i];
            }
            const int l = V::cross(sum, goal, lane);
            int at = 0;
            bool past = false;
#pragma unroll
            for (int i = 0; i < NE; i++) {
                const long long n = __shfl_sync(0xffffffffu, part[i], l);
                if (n > 0 && !past) {
                    at = i;
                    past = n > goal;
                    if (!past && goal != LLONG_MAX) goal -= n;
                }
            }
            if (!past) goal = LLONG_MAX;
            finder = min(l * each + at, ctas * kWarps - 1);
        }
    }
    if (lane == 0) {
        p.n_accepted[b] = count;
        if (finder < 0) p.next_token[b] = -1;
    }
#pragma unroll
    for (int j = 0; j < 2; j++)
        if (lane + 32 * j < p.max_q) p.path[(int64_t)b * p.max_q + lane + 32 * j] = place[j];
    give(0, 0, Pair(), 0, 0, finder, whole, goal);
}

template <bool F32, bool DRAFT, int kWarps> cudaError_t run_warps(const VerifyParams &p, int ctas, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_seq * ctas));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<F32, DRAFT, kWarps>, p, ctas);
}
// 16 warps per CTA, two CTAs per SM, while all clusters are resident together that way (with one CTA per SM a GPU's clusters of
// 8 leave SMs over: 16 of them took 17 us instead of 11); else 8 warps, four CTAs per SM (64 sequences: 44 us, 48 with 16).
template <bool F32, bool DRAFT> cudaError_t run(const VerifyParams &p, int ctas, int sms, cudaStream_t s, bool pdl)
{
    return 2 * (int64_t)p.n_seq * ctas <= 3 * sms ? run_warps<F32, DRAFT, 16>(p, ctas, s, pdl) : run_warps<F32, DRAFT, 8>(p, ctas, s, pdl);
}

}  // namespace

cudaError_t launch_verify(VerifyParams p, int x_f32, int sms, cudaStream_t s, bool pdl)
{
    if (cudaError_t e = device_error_word(&p.error)) return e;
    int ctas = 1;
    while (ctas < kMaxCtas && (int64_t)ctas * kLeast < p.vocab) ctas *= 2;
    return x_f32 ? (p.draft ? run<true, true>(p, ctas, sms, s, pdl) : run<true, false>(p, ctas, sms, s, pdl))
                 : (p.draft ? run<false, true>(p, ctas, sms, s, pdl) : run<false, false>(p, ctas, sms, s, pdl));
}

}  // namespace bqg
