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
//  * A cluster of up to 8 CTAs takes a sequence, each a contiguous part of the row.  The first one walks the tree and gives the
//    others their orders (a sum, or the end) through shared memory, two cluster barriers each: who arrives how
//    often is decided in one place.
//  * An answer is a whole number and depends on where a sum of up to 2^18 terms crosses a border, so fp32 sums (off by 1e-7:
//    another token once in some hundred draws) would not do, and fp64's rate is 1/64 of fp32's here: p - c q is
//    formed as an fp32 pair with the products' and the difference's errors, and added with error-free sums:
//    about 2^-45 of the sum.  The few numbers of the walk itself are fp64.
//  * The crossing is looked for in the sums of CTAs, of warps (contiguous ranges), then in the warp's range, which one
//    warp reads again: first lane by lane, then token by token.
#include <cooperative_groups.h>

#include "bqg_verify.cuh"

namespace bqg {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCtas = 8, kMaxDrafts = 64;
constexpr int kLeast = 2048;           // values of a row that a CTA is taken for

// An unevaluated sum of two fp32 numbers.
struct Pair {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float h, float l)
    {
        float e;
        two_sum(hi, h, hi, e);
        lo = __fadd_rn(lo, __fadd_rn(e, l));
    }
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

struct Order {
    int sum;                           // 0: the end
    int row;                           // of target and draft
    float c_hi, c_lo;                  // what q is taken off with
    int n_gone;                        // chosen drafts that were rejected here
    int gone[kMaxDrafts];
};

// A probability: what is no positive number counts as none.
__device__ __forceinline__ float prob(float x) { return x > 0.f && x < __int_as_float(0x7f800000) ? x : 0.f; }
template <bool F32> __device__ __forceinline__ float load_prob(const void *x, int64_t i)
{
    if constexpr (F32) return prob(__ldg(reinterpret_cast<const float *>(x) + i));
    else return prob(__uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(x) + i) << 16));
}

// What is left of p after c q: a pair, (0, 0) if it is not positive.
__device__ __forceinline__ void rest(float p, float q, float ch, float cl, float &hi, float &lo)
{
    const float m = __fmul_rn(q, ch);
    const float me = __fadd_rn(fmaf(q, ch, -m), __fmul_rn(q, cl));
    float e;
    two_sum(p, -m, hi, e);
    lo = __fsub_rn(e, me);
    if (!(__fadd_rn(hi, lo) > 0.f)) hi = lo = 0.f;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

template <bool F32, bool DRAFT> struct Verify {
    // r at token x < vocab of the order's row.
    static __device__ __forceinline__ void left(const VerifyParams &p, const Order &o, int64_t t0, int64_t q0, int x, unsigned long long gone,
                                                float &hi, float &lo)
    {
        hi = load_prob<F32>(p.target, t0 + x);
        lo = 0.f;
        if constexpr (DRAFT) {
            if (o.c_hi > 0.f) rest(hi, load_prob<F32>(p.draft, q0 + x), o.c_hi, o.c_lo, hi, lo);
        } else {
            for (; gone; gone &= gone - 1)
                if (o.gone[__ffsll(gone) - 1] == x) hi = 0.f;
        }
    }
    // Which of the rejected tokens lie in [a, e).
    static __device__ __forceinline__ unsigned long long gone_in(const Order &o, int a, int e, int lane)
    {
        if (DRAFT) return 0;
        const bool lo = lane < o.n_gone && o.gone[lane] >= a && o.gone[lane] < e;
        const bool hi = lane + 32 < o.n_gone && o.gone[lane + 32] >= a && o.gone[lane + 32] < e;
        return (unsigned long long)__ballot_sync(0xffffffffu, lo) | (unsigned long long)__ballot_sync(0xffffffffu, hi) << 32;
    }
    // The sum of r over tokens a .. e - 1, in all lanes.
    static __device__ __forceinline__ Pair sum(const VerifyParams &p, const Order &o, int a, int e, int lane)
    {
        const int64_t t0 = (int64_t)o.row * p.target_stride, q0 = (int64_t)o.row * p.draft_stride;
        const unsigned long long gone = gone_in(o, a, e, lane);
        constexpr int U = 8;
        Pair acc[2];
        for (int x0 = a; x0 < e; x0 += 32 * U) {
            float pv[U], qv[U];
#pragma unroll
            for (int i = 0; i < U; i++) {
                const int x = x0 + 32 * i + lane;
                pv[i] = x < e ? load_prob<F32>(p.target, t0 + x) : 0.f;
                if constexpr (DRAFT) qv[i] = x < e && o.c_hi > 0.f ? load_prob<F32>(p.draft, q0 + x) : 0.f;
            }
            if (!DRAFT && gone) {
#pragma unroll
                for (int i = 0; i < U; i++)
                    for (unsigned long long g = gone; g; g &= g - 1)
                        if (o.gone[__ffsll(g) - 1] == x0 + 32 * i + lane) pv[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < U; i++) {
                float hi = pv[i], lo = 0.f;
                if constexpr (DRAFT) rest(pv[i], qv[i], o.c_hi, o.c_lo, hi, lo);
                acc[i & 1].add(hi, lo);
            }
        }
        acc[0].add(acc[1].hi, acc[1].lo);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1)
            acc[0].add(__shfl_xor_sync(0xffffffffu, acc[0].hi, s), __shfl_xor_sync(0xffffffffu, acc[0].lo, s));
        return acc[0];
    }
    // The first of 32 consecutive parts (this lane's: v) whose running sum from `base` on exceeds `goal`; without one,
    // which is a matter of rounding, the last part that is not nothing; -1: all are.  base: the sum before it, or of all.
    static __device__ __forceinline__ int cross(double v, double goal, int lane, double &base)
    {
        double run = v;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, run, s);
            if (lane >= s) run += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + run > goal), some = __ballot_sync(0xffffffffu, v > 0.0);
        const int at = past & some ? __ffs(past & some) - 1 : -1;
        const double before = __shfl_sync(0xffffffffu, run - v, at < 0 ? 0 : at), all = __shfl_sync(0xffffffffu, run, 31);
        if (at < 0) {
            base += all;
            return -1;
        }
        base += before;
        return at;
    }
    // ... among tokens a .. e - 1, at least one of which has something left.
    static __device__ int token(const VerifyParams &p, const Order &o, int a, int e, double base, double goal, int lane)
    {
        const int64_t t0 = (int64_t)o.row * p.target_stride, q0 = (int64_t)o.row * p.draft_stride;
        const unsigned long long gone = gone_in(o, a, e, lane);
        const int per = (e - a + 31) / 32, b = min(a + lane * per, e), n = min(per, e - b);
        Pair s;
#pragma unroll 4
        for (int i = 0; i < n; i++) {
            float hi, lo;
            left(p, o, t0, q0, b + i, gone, hi, lo);
            s.add(hi, lo);
        }
        const double v = s.value();
        int l = cross(v, goal, lane, base);
        if (l < 0) {
            l = 31 - __clz(__ballot_sync(0xffffffffu, v > 0.0) | 1u);
            goal = __longlong_as_double(0x7ff0000000000000ll);         // its last token
        }
        const int first = __shfl_sync(0xffffffffu, b, l), count = __shfl_sync(0xffffffffu, n, l);
        int last = first;
        for (int i = 0; i < count; i += 32) {
            float hi = 0.f, lo = 0.f;
            if (i + lane < count) left(p, o, t0, q0, first + i + lane, gone, hi, lo);
            const double r = (double)hi + (double)lo;
            const int at = cross(r, goal, lane, base);
            if (at >= 0) return first + i + at;
            const unsigned some = __ballot_sync(0xffffffffu, r > 0.0);
            if (some) last = first + i + 31 - __clz(some);
        }
        return last;
    }
};

template <bool F32, bool DRAFT>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p, int ctas)
{
    namespace cg = cooperative_groups;
    using V = Verify<F32, DRAFT>;
    __shared__ Order order;
    __shared__ Pair warp_sum[kWarps];
    __shared__ double cta_sum;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % ctas, b = blockIdx.x / ctas;
    const bool walker = rank == 0 && warp == 0;
    pdl_wait();
    pdl_launch_dependents();

    // values of a row per warp, a multiple of 32
    const int per = (int)((((int64_t)p.vocab + ctas * kWarps - 1) / (ctas * kWarps) + 31) & ~31ll);
    auto range = [&](int cta, int w, int &a, int &e) {
        a = (int)min((int64_t)(cta * kWarps + w) * per, (int64_t)p.vocab);
        e = (int)min((int64_t)a + per, (int64_t)p.vocab);
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
        if (!order.sum) return false;
        int a, e;
        range(rank, warp, a, e);
        const Pair s = V::sum(p, order, a, e, lane);
        if (lane == 0) warp_sum[warp] = s;
        __syncthreads();
        if (warp == 0) {
            Pair t;
            if (lane < kWarps) t = warp_sum[lane];
#pragma unroll
            for (int i = kWarps / 2; i > 0; i >>= 1) t.add(__shfl_xor_sync(0xffffffffu, t.hi, i), __shfl_xor_sync(0xffffffffu, t.lo, i));
            if (lane == 0) cta_sum = t.value();
        }
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
    int up[2], tok[2];
    float u[2], pt[2], qt[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int i = lane + 32 * j;
        up[j] = tok[j] = -1;
        u[j] = pt[j] = 0.f;
        qt[j] = 1.f;
        if (i >= T) continue;
        u[j] = p.u[q0 + i];
        if (i == 0) continue;
        tok[j] = p.tokens[q0 + i];
        up[j] = p.parent ? p.parent[q0 + i] : i - 1;
        if (up[j] < 0 || up[j] >= i || tok[j] < 0 || tok[j] >= p.vocab) {
            bad |= BQG_DEVERR_DRAFT;
            up[j] = -1;
            continue;
        }
        const int64_t row = q0 + up[j];
        pt[j] = load_prob<F32>(p.target, row * p.target_stride + tok[j]);
        if constexpr (DRAFT) qt[j] = load_prob<F32>(p.draft, row * p.draft_stride + tok[j]);
    }
    if (bad) atomicOr(p.error, bad);
    __syncwarp();
    if (ctas > 1) cluster_wait();
    auto pick = [&](auto (&v)[2], int i) {
        const auto lo = __shfl_sync(0xffffffffu, v[0], i & 31), hi = __shfl_sync(0xffffffffu, v[1], i & 31);
        return i < 32 ? lo : hi;
    };
    auto give = [&](int sum, int64_t row, double c, int n_gone) {
        __syncwarp();
        if (lane < ctas) {                                // to one CTA per lane
            Order *o = ctas > 1 ? cluster.map_shared_rank(&order, lane) : &order;
            o->sum = sum;
            o->row = (int)row;
            o->c_hi = (float)c;
            o->c_lo = (float)(c - (double)(float)c);
            o->n_gone = n_gone;
            if (lane)
                for (int i = 0; i < n_gone; i++) o->gone[i] = order.gone[i];
        }
        __syncwarp();
        round();
        double z = 0.0;                                   // the CTAs' sums, in their order: one per lane
        if (sum && lane < ctas) z = ctas > 1 ? *cluster.map_shared_rank(&cta_sum, lane) : cta_sum;
        return z;
    };
    auto all_of = [&](double z) {
#pragma unroll
        for (int s = 4; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
        return __shfl_sync(0xffffffffu, z, 0);
    };
    int node = 0, count = T > 0, place[2] = {lane == 0 && T > 0 ? 0 : -1, -1}, next = -1;   // place: of the path
    if (T > 0) {
        int last = 0, n_gone = 0;                         // the last draft looked at
        double Z = 1.0, c = 0.0, parts = 0.0;
        bool known = false;                               // `parts` and the warps' sums are those of r
        for (;;) {
            unsigned long long below = (unsigned long long)__ballot_sync(0xffffffffu, up[0] == node) |
                                       (unsigned long long)__ballot_sync(0xffffffffu, up[1] == node) << 32;
            below &= last < 63 ? ~0ull << (last + 1) : 0ull;
            if (!below) break;
            const int i = __ffsll(below) - 1;
            last = i;
            const double ui = pick(u, i), qi = pick(qt, i);
            double pi = pick(pt, i);
            const int ti = pick(tok, i);
            bool yes;
            if constexpr (DRAFT) {
                const double l = pi - c * qi;
                yes = ui * qi * Z < (l > 0.0 ? l : 0.0);
            } else {
                const bool again = (lane < n_gone && order.gone[lane] == ti) || (lane + 32 < n_gone && order.gone[lane + 32] == ti);
                if (__any_sync(0xffffffffu, again)) pi = 0.0;
                yes = ui * Z < pi;
            }
            if (yes) {
                node = i;
                if (lane == (count & 31)) place[count >> 5] = i;
                count++;
                Z = 1.0;
                c = 0.0;
                n_gone = 0;
                known = false;
            } else if constexpr (DRAFT) {
                c += Z;
                parts = give(1, q0 + node, c, 0);
                Z = all_of(parts);
                known = true;
            } else {
                Z -= pi;
                if (lane == 0) order.gone[n_gone] = ti;
                n_gone++;
                __syncwarp();
            }
        }
        if (!known) {
            parts = give(1, q0 + node, 0.0, n_gone);
            Z = all_of(parts);
        }
        if (!(Z > 0.0) && (known || n_gone)) {            // nothing left: the target's own
            parts = give(1, q0 + node, 0.0, 0);
            Z = all_of(parts);
        }
        if (Z > 0.0) {
            const double goal = (double)__shfl_sync(0xffffffffu, u[0], 0) * Z;
            double base = 0.0;
            double far = goal;
            int cta = V::cross(parts, far, lane, base);
            if (cta < 0) {
                cta = 31 - __clz(__ballot_sync(0xffffffffu, parts > 0.0) | 1u);
                far = __longlong_as_double(0x7ff0000000000000ll);
            }
            const Pair *sums = ctas > 1 ? cluster.map_shared_rank(warp_sum, cta) : warp_sum;
            const double w = lane < kWarps ? sums[lane].value() : 0.0;
            int at = V::cross(w, far, lane, base);
            if (at < 0) {
                at = 31 - __clz(__ballot_sync(0xffffffffu, w > 0.0) | 1u);
                far = __longlong_as_double(0x7ff0000000000000ll);
            }
            int a, e;
            range(cta, at, a, e);
            if (a < e) next = V::token(p, order, a, e, base, far, lane);
        }
    }
    if (lane == 0) {
        p.n_accepted[b] = count;
        p.next_token[b] = next;
    }
#pragma unroll
    for (int j = 0; j < 2; j++)
        if (lane + 32 * j < p.max_q) p.path[(int64_t)b * p.max_q + lane + 32 * j] = place[j];
    give(0, 0, 0.0, 0);
}

template <bool F32, bool DRAFT> cudaError_t run(const VerifyParams &p, int ctas, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_seq * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<F32, DRAFT>, p, ctas);
}

}  // namespace

cudaError_t launch_verify(VerifyParams p, int x_f32, cudaStream_t s, bool pdl)
{
    if (cudaError_t e = device_error_word(&p.error)) return e;
    int ctas = 1;
    while (ctas < kMaxCtas && (int64_t)ctas * kLeast < p.vocab) ctas *= 2;
    return x_f32 ? (p.draft ? run<true, true>(p, ctas, s, pdl) : run<true, false>(p, ctas, s, pdl))
                 : (p.draft ? run<false, true>(p, ctas, s, pdl) : run<false, false>(p, ctas, s, pdl));
}

}  // namespace bqg
