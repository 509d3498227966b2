// verify.hip -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// With p_t and q_t the target's and the drafting model's probabilities, drafts
// x_t are accepted one after another while u_t q_t(x_t) < p_t(x_t).  At the
// first that is not, a token is drawn from max(p_t - q_t, 0), and behind the
// last one, if all are, from p_t: the first v whose cumulative mass exceeds
// u_last times the whole.
//
// Whole numbers come out of comparisons of sums over the vocabulary, so all of
// it is in fp64, the exponentials too (a polynomial of 2^f, relative error
// 2e-12): in fp32 one draw in some hundred would fall on the other side of a
// border.  Two launches: the largest logit and the sum of every row, in one pass
// over all logits; then the mass of pieces of the one row of each sequence that
// is drawn from (every workgroup finds out which by itself: a few comparisons),
// and, in the workgroup that is the last of its sequence, the search over pieces
// and inside one.
//
// 64 sequences of 4 drafts over 131072 tokens bf16: 59 us for the sums (2.5 TB/s;
// fp64 operations bound them) and 40 for the rest, half of it trips to memory one
// after another; one sequence over 50280 fp32: 6 and 14 us.
#include <cfloat>
#include <type_traits>

#include "device_common.h"
#include "dpp64.h"
#include "lm_internal.h"
#include "msscan_internal.h"

namespace msscan {
namespace verify {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kMine = 8;  // values a thread looks at together in the search
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef u4 u4_align2 __attribute__((aligned(2)));
typedef u4 u4_align4 __attribute__((aligned(4)));

// 2^x for x <= 0 (or NaN); 0 from -1000 down, which no sum notices.  power(): of
// either sign, up to 1000.
__device__ __forceinline__ double exp2_64(double x) {
    const double n = __builtin_rint(x), f = (x - n) * 0.693147180559945309417;
    // the series of e^f, |f| <= 0.3466: the first term left out is 2e-13
    double p = 1.0 / 3628800.0;
    p = fma(p, f, 1.0 / 362880.0);
    p = fma(p, f, 1.0 / 40320.0);
    p = fma(p, f, 1.0 / 5040.0);
    p = fma(p, f, 1.0 / 720.0);
    p = fma(p, f, 1.0 / 120.0);
    p = fma(p, f, 1.0 / 24.0);
    p = fma(p, f, 1.0 / 6.0);
    p = fma(p, f, 0.5);
    p = fma(p, f, 1.0);
    p = fma(p, f, 1.0);
    const double y = __builtin_amdgcn_ldexp(p, (int)n);
    return x < -1000.0 ? 0.0 : y;
}

__device__ __forceinline__ double power(double x) {
    return x > 0.0 ? 1.0 / exp2_64(-x) : exp2_64(x);
}

// The same for a whole vocabulary, with the 128th roots of 2 in LDS: half the
// fp64 operations, which run at half fp32's rate here and bound the sums of rows
// (64 x 9 rows of 131072 bf16: 80 -> 56 us).  x = n / 128 + r, |r| <= 1/256; the
// series of 2^r up to r^3, whose next term is 2e-12.  The addition of 3 2^44
// leaves n in the low bits.
struct Roots {
    double v[128];
    __device__ __forceinline__ void make() {
        if (threadIdx.x < 128) v[threadIdx.x] = exp2_64((double)threadIdx.x / 128.0 - 1.0) * 2.0;
    }
    // |x| up to 2000 (or NaN)
    __device__ __forceinline__ double exp2(double x) const {
        const double magic = 52776558133248.0;
        const double shifted = x + magic, r = x - (shifted - magic);
        const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, shifted);
        double p = 0.0555041086648215800;
        p = fma(p, r, 0.2402265069591007123);
        p = fma(p, r, 0.6931471805599453094);
        p = fma(p, r, 1.0);
        return __builtin_amdgcn_ldexp(p * v[n & 127], n >> 7);
    }
    // any x up to 2000: 2^-999 (beside what reaches 1, nothing) or 0 from -999 down
    __device__ __forceinline__ double exp2_above(double x) const {
        return exp2(x < -999.0 ? -999.0 : x);
    }
    __device__ __forceinline__ double exp2_or_0(double x) const {
        const double y = exp2_above(x);
        return x < -999.0 ? 0.0 : y;
    }
};

// Exponents of logits, in base 2, are v c with c the scale times log2 e.  A product
// by itself: part of a fused one, it would be another number than the m that a sum
// stands beside.
__device__ __forceinline__ double exponent(float v, double c) {
#pragma clang fp contract(off)
    return (double)v * c;
}

// The exponent of a logit over m, the rounded exponent of one of the row's (or of
// a part's).  The fused product takes v c as it is, so weights are right beside m to
// 2^-53 of their own exponents, however large m.  m's rounding then shows as a
// factor that all weights share, 2^(v c - m) of the logit that m is of.  From
// |m| = 2^50 on it would reach 2^-3 and more of an exponent, and leave fp64's range
// at rows of the type's lowest value; but there neighbouring logits are 2^25 apart,
// and a smaller c that is a power of two, in which products are exact, gives what
// the full one does: 1 for the same logit, and 0 below it.
struct Over {
    double c, m;
    __device__ __forceinline__ Over() = default;
    __device__ __forceinline__ Over(double m_, double c_) : c(c_), m(m_) {
        if (fabs(m_) >= 0x1p50 && fabs(m_) < INFINITY) {
            c = __builtin_amdgcn_ldexp(1.0, __builtin_amdgcn_frexp_exp(c_) - 1);
            m = exponent((float)(m_ / c_), c);  // the logit itself: fp32 rounds 2^-52 away
        }
    }
    __device__ __forceinline__ double operator()(float v) const { return fma((double)v, c, -m); }
};

// An exponent (in base 2) near the largest, and the sum beside it.  Nothing yet,
// or only masked logits: m = -inf, s = 0.  NaN and +inf: s becomes NaN.
struct Sum {
    double m, s;
    __device__ __forceinline__ void add(const Sum& o) {
        if (o.m > m) {
            s = (m == -INFINITY ? s : s * exp2_64(m - o.m)) + o.s;
            m = o.m;
        } else {
            s += o.m == -INFINITY ? o.s : o.s * exp2_64(o.m - m);
        }
    }
};

template <bool BF16>
struct Row {
    static constexpr int W = BF16 ? 8 : 4;
    typedef typename std::conditional<BF16, uint16_t, float>::type E;
    typedef typename std::conditional<BF16, u4_align2, u4_align4>::type U;
    // W values from place i on of n; -inf behind the end
    static __device__ __forceinline__ void load(const void* row, int64_t i, int64_t n,
                                                float (&v)[W]) {
        const E* p = static_cast<const E*>(row) + i;
        if (i + W <= n) {
            const u4 x = *reinterpret_cast<const U*>(p);
#pragma unroll
            for (int e = 0; e < W; ++e)
                if constexpr (BF16)
                    v[e] = __uint_as_float(e & 1 ? x[e / 2] & 0xffff0000u : x[e / 2] << 16);
                else
                    v[e] = __uint_as_float(x[e]);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = i + e < n ? ld<BF16>(p, e) : -INFINITY;
        }
    }
};

template <bool BF16>
__device__ __forceinline__ const void* row_of(const VerifyArgs& a, int64_t r) {
    constexpr int size = BF16 ? 2 : 4;
    const int64_t own = (int64_t)a.batch * (a.drafts + 1);
    return r < own ? static_cast<const char*>(a.logits) + r * a.ld * size
                   : static_cast<const char*>(a.draft_logits) + (r - own) * a.ldd * size;
}

// ---- sums of rows ------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(VerifyArgs a) {
    constexpr int W = Row<BF16>::W;
    __shared__ Sum sums[kThreads / 64];
    __shared__ Roots roots;
    roots.make();
    __syncthreads();
    const int64_t r = blockIdx.x / a.splits;
    const int split = blockIdx.x % a.splits;
    const int64_t i0 = split * a.per, i1 = i0 + a.per < a.V ? i0 + a.per : a.V;
    const void* row = row_of<BF16>(a, r);
    const double c = (double)a.scale * 1.4426950408889634074;
    // Sums stand beside 2^m of a logit met early on.  fp64 reaches far enough that
    // only one 2^400 times as likely (800, where fp32's next logit is that far) calls
    // for another; and 2^-999 of it is nothing.  The borders are fp32 and may be the
    // logit itself, so what lies below `low` is looked at by its exponent.
    float high = -INFINITY, low = INFINITY;
    Over over{};
    double m = -INFINITY, s = 0.0;
    for (int64_t i = i0 + threadIdx.x * W; i < i1; i += kThreads * W) {
        float v[W];
        Row<BF16>::load(row, i, i1, v);
        float t = v[0], l = v[0];
#pragma unroll
        for (int e = 1; e < W; ++e) t = fmaxf(t, v[e]), l = fminf(l, v[e]);
        if (t > high) {
            const double now = exponent(t, c);
            s = m == -INFINITY ? s : s * exp2_64(m - now);
            m = now;
            over = Over(m, c);
            high = (float)((over.m + 400.0) / over.c);
            low = fmaxf((float)((over.m - 999.0) / over.c), -FLT_MAX);  // above -inf
        }
        if (m == -INFINITY) {  // nothing but masked logits, or NaN
#pragma unroll
            for (int e = 0; e < W; ++e) s += v[e] == v[e] ? 0.0 : (double)v[e];
            continue;
        }
        if (l < low) {
#pragma unroll
            for (int e = 0; e < W; ++e) s += roots.exp2_above(over(v[e]));
            continue;
        }
#pragma unroll
        for (int e = 0; e < W; ++e) s += roots.exp2(over(v[e]));
    }
    if (split == 0 && r < a.batch) {  // for the next launch
        if (threadIdx.x == 0) a.done[r] = 0;
        for (int n = threadIdx.x; n < 2 * a.pieces; n += kThreads)
            a.mass[r * a.pieces * 2 + n] = -1.0;
    }
    Sum x{m, s};
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x.add(Sum{__shfl_xor(x.m, d), __shfl_xor(x.s, d)});
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 64; ++w) x.add(sums[w]);
        a.part[blockIdx.x * 2] = x.m;
        a.part[blockIdx.x * 2 + 1] = x.s;
    }
}

// ---- which drafts are accepted --------------------------------------------------------
struct Shared {
    Sum p[kMaxDrafts + 1], q[kMaxDrafts];
    int yes[kMaxDrafts];
    double x[kMaxDrafts];  // the drafts' exponents over their rows' m
    int count;
};

__device__ __forceinline__ double wave_sum(double x) { return lane64(scan64(x), 63); }
// A row's parts, one after another by a thread, or by the lanes of a wave.
__device__ __forceinline__ Sum row_sum(const VerifyArgs& a, int64_t r) {
    Sum x{-INFINITY, 0.0};
    for (int n = 0; n < a.splits; ++n)
        x.add(Sum{a.part[(r * a.splits + n) * 2], a.part[(r * a.splits + n) * 2 + 1]});
    return x;
}
__device__ __forceinline__ Sum row_sum_by_wave(const VerifyArgs& a, int64_t r) {
    const int n = threadIdx.x & 63;
    Sum x{-INFINITY, 0.0};
    if (n < a.splits) x = Sum{a.part[(r * a.splits + n) * 2], a.part[(r * a.splits + n) * 2 + 1]};
    double m = x.m;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double y = __shfl_xor(m, d);
        m = y > m ? y : m;
    }
    return {m, wave_sum(m == -INFINITY ? x.s : x.s * exp2_64(x.m - m))};
}
// whether the row is a distribution
__device__ __forceinline__ bool proper(const Sum& x) { return x.s > 0.0 && x.s < INFINITY; }

__device__ __forceinline__ int64_t draft(const VerifyArgs& a, int b, int t) {
    const int64_t i = (int64_t)b * a.drafts + t;
    return a.wide ? static_cast<const int64_t*>(a.tokens_in)[i]
                  : static_cast<const int32_t*>(a.tokens_in)[i];
}

template <bool BF16>
__device__ __forceinline__ void decide(const VerifyArgs& a, int b, Shared& sh) {
    const int T = a.drafts, t = threadIdx.x;
    const int64_t first = (int64_t)b * (T + 1);
    const int64_t first_q = (int64_t)a.batch * (T + 1) + (int64_t)b * T;
    // the drafts' own logits are on their way while the rows' sums are joined
    int64_t v = -1;
    float u = 0.f, xp = 0.f, xq = 0.f;
    if (t < T) {
        v = draft(a, b, t);
        u = a.uniforms[first + t];
        if (v >= 0 && v < a.V) {
            xp = ld<BF16>(row_of<BF16>(a, first + t), v);
            if (a.draft_logits) xq = ld<BF16>(row_of<BF16>(a, first_q + t), v);
        } else {
            v = -1;
        }
    }
    if (a.splits > 4) {
        for (int n = t >> 6; n <= T + (a.draft_logits ? T : 0); n += kThreads / 64) {
            const Sum x = row_sum_by_wave(a, n <= T ? first + n : first_q + n - T - 1);
            if ((t & 63) == 0) (n <= T ? sh.p[n] : sh.q[n - T - 1]) = x;
        }
    } else if (t <= T) {
        sh.p[t] = row_sum(a, first + t);
    } else if (t >= 128 && t - 128 < T && a.draft_logits) {
        sh.q[t - 128] = row_sum(a, first_q + t - 128);
    }
    __syncthreads();
    if (t < T) {
        const double c = (double)a.scale * 1.4426950408889634074;
        bool yes = false;
        if (v >= 0 && proper(sh.p[t])) {
            const double x = Over(sh.p[t].m, c)(xp);
            const double p = power(x) / sh.p[t].s;
            double q = 1.0;
            if (a.draft_logits)
                q = proper(sh.q[t]) ? power(Over(sh.q[t].m, c)(xq)) / sh.q[t].s : INFINITY;
            yes = (double)u * q < p;
            sh.x[t] = x;
        }
        sh.yes[t] = yes;
    }
    __syncthreads();
    if (t == 0) {
        int n = 0;
        while (n < T && sh.yes[n]) ++n;
        sh.count = n;
    }
    __syncthreads();
}

// What is drawn from: the mass that is left of the target's at place v, and the
// target's own (in units of its largest).
struct Left {
    double p, left;
};
template <bool BF16>
struct Drawn {
    const void *prow, *qrow;
    Sum p, q;
    Over over_p, over_q;
    double ratio;  // of what a unit of q's row is worth in p's
    int64_t one;   // a draft without probabilities of its own
    __device__ __forceinline__ Drawn(const VerifyArgs& a, int b, const Shared& sh) {
        const int n = sh.count, T = a.drafts;
        const double c = (double)a.scale * 1.4426950408889634074;
        prow = row_of<BF16>(a, (int64_t)b * (T + 1) + n);
        p = sh.p[n];
        over_p = Over(p.m, c);
        qrow = nullptr;
        one = -1;
        if (n < T) {
            if (!a.draft_logits) {
                one = draft(a, b, n);
            } else if (proper(sh.q[n])) {
                qrow = row_of<BF16>(a, (int64_t)a.batch * (T + 1) + (int64_t)b * T + n);
                q = sh.q[n];
                over_q = Over(q.m, c);
                ratio = p.s / q.s;
            }
        }
    }
    __device__ __forceinline__ Left at(const Roots& roots, float x, float y, int64_t v) const {
        const double mine = roots.exp2_or_0(over_p(x));
        double left = mine;
        if (qrow) left = fma(-roots.exp2_or_0(over_q(y)), ratio, mine);
        if (v == one) left = 0.0;
        return {mine, left > 0.0 ? left : 0.0};
    }
};

// Sums up to and with each thread's x, over the workgroup.
__device__ __forceinline__ double scan(double x, double (&sums)[kThreads / 64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    x = scan64(x);
    __syncthreads();
    if (lane == 63) sums[wave] = x;
    __syncthreads();
    for (int w = 0; w < wave; ++w) x += sums[w];
    return x;
}

// Of the workgroup's threads whose x is not negative, in order, the first one's
// x, or the last one's; or -1.
__device__ __forceinline__ int of_waves(int x, bool last, int (&of)[kThreads / 64]) {
    const uint64_t in = __ballot(x >= 0);
    int mine = -1;
    if (in) mine = __builtin_amdgcn_readlane(x, last ? 63 - __builtin_clzll(in) : __builtin_ctzll(in));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) of[threadIdx.x >> 6] = mine;
    __syncthreads();
    int r = -1;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w)
        if (of[w] >= 0 && (last || r < 0)) r = of[w];
    return r;
}

// A mass that another workgroup wrote in this launch.  It is one word, which no
// fence has to order (a fence would write back and drop whole caches: 50 of 76 us
// for 64 sequences); at most it is still on its way, for who reads it has seen
// that its writer was past writing it.
__device__ __forceinline__ double shared_load(const double* p) {
    double x;
    do {
        x = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } while (x < 0.0);
    return x;
}

// The token drawn, or -1: over the pieces' masses, then inside one.
template <bool BF16>
__device__ __forceinline__ int64_t draw(const VerifyArgs& a, int b, const Drawn<BF16>& from,
                                        const Roots& roots) {
    __shared__ double sums[kThreads / 64];
    __shared__ int of[kThreads / 64];
    __shared__ double before;  // mass ahead of the piece
    constexpr int W = Row<BF16>::W;
    const int tid = threadIdx.x;
    const double* mass = a.mass + (int64_t)b * a.pieces * 2;
    // the whole: of what is left, or of the target's where nothing is
    double whole = 0.0;
    int which = 0;
    for (; which < 2; ++which) {
        double x = 0.0;
        for (int n = tid; n < a.pieces; n += kThreads) x += shared_load(mass + n * 2 + which);
        x = wave_sum(x);
        __syncthreads();
        if ((tid & 63) == 0) sums[tid >> 6] = x;
        __syncthreads();
        whole = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        if (whole > 0.0) break;
    }
    if (!proper(from.p) || !(whole > 0.0)) return -1;
    const double border = (double)a.uniforms[(int64_t)b * (a.drafts + 1) + a.drafts] * whole;
    // the first piece past the border, or else (rounding, or a number that is not
    // below 1) the last one with mass at all
    int piece = -1, last = -1;
    double ahead = 0.0;
    for (int n0 = 0; n0 < a.pieces && piece < 0; n0 += kThreads) {
        const int n = n0 + tid;
        const double x = n < a.pieces ? shared_load(mass + n * 2 + which) : 0.0;
        const double upto = ahead + scan(x, sums);
        ahead += (sums[0] + sums[1]) + (sums[2] + sums[3]);
        piece = of_waves(x > 0.0 && upto > border ? n : -1, false, of);
        last = max(last, of_waves(x > 0.0 ? n : -1, true, of));
        if (n == piece) before = upto - x;
    }
    const bool over = piece < 0;
    if (over) piece = last;
    __syncthreads();
    const int64_t i0 = (int64_t)piece * a.piece, i1 = i0 + a.piece < a.V ? i0 + a.piece : a.V;
    ahead = over ? 0.0 : before;
    last = -1;
    for (int64_t j0 = i0; j0 < i1; j0 += kThreads * kMine) {
        // kMine neighbouring values a thread
        double x[kMine], sum = 0.0;
        const int mine = tid * kMine;
#pragma unroll
        for (int k = 0; k < kMine; k += W) {
            float u[W], v[W];
            Row<BF16>::load(from.prow, j0 + mine + k, i1, u);
            if (from.qrow) Row<BF16>::load(from.qrow, j0 + mine + k, i1, v);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const Left l = from.at(roots, u[e], from.qrow ? v[e] : 0.f, j0 + mine + k + e);
                x[k + e] = which ? l.p : l.left;
                sum += x[k + e];
            }
        }
        double upto = ahead + (scan(sum, sums) - sum);
        ahead += (sums[0] + sums[1]) + (sums[2] + sums[3]);
        int found = -1, mass_at = -1;
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            upto += x[e];
            if (x[e] > 0.0) {
                mass_at = mine + e;
                if (found < 0 && !over && upto > border) found = mine + e;
            }
        }
        found = of_waves(found, false, of);
        if (found >= 0) return j0 + found;
        mass_at = of_waves(mass_at, true, of);
        if (mass_at >= 0) last = (int)(j0 - i0) + mass_at;
    }
    return i0 + last;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a) {
    constexpr int W = Row<BF16>::W;
    __shared__ Shared sh;
    __shared__ Roots roots;
    __shared__ double sums[2][kThreads / 64];
    __shared__ bool finish;
    const int b = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces;
    const int tid = threadIdx.x, T = a.drafts;
    roots.make();
    decide<BF16>(a, b, sh);
    const Drawn<BF16> from(a, b, sh);
    const int64_t i0 = (int64_t)piece * a.piece, i1 = i0 + a.piece < a.V ? i0 + a.piece : a.V;
    double left = 0.0, own = 0.0;
    if (proper(from.p))
#pragma unroll 2
        for (int64_t i = i0 + tid * W; i < i1; i += kThreads * W) {
            float x[W], y[W];
            Row<BF16>::load(from.prow, i, i1, x);
            if (from.qrow) Row<BF16>::load(from.qrow, i, i1, y);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const Left l = from.at(roots, x[e], from.qrow ? y[e] : 0.f, i + e);
                left += l.left;
                own += l.p;
            }
        }
    left = wave_sum(left);
    own = wave_sum(own);
    if ((tid & 63) == 0) {
        sums[0][tid >> 6] = left;
        sums[1][tid >> 6] = own;
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
            __hip_atomic_store(a.mass + (int64_t)blockIdx.x * 2 + n,
                               (sums[n][0] + sums[n][1]) + (sums[n][2] + sums[n][3]),
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        finish = __hip_atomic_fetch_add(a.done + b, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.pieces - 1;
    }
    __syncthreads();
    if (!finish) return;
    const int64_t drawn = draw<BF16>(a, b, from, roots);
    // the tokens, and their log probabilities under the target
    if (tid <= T) {
        const int64_t at = (int64_t)b * (T + 1) + tid;
        int64_t v = -1;
        if (tid < sh.count) v = draft(a, b, tid);
        else if (tid == sh.count) v = drawn;
        double lp = 0.0;
        if (v >= 0) {
            const double x = tid < sh.count ? sh.x[tid]
                                            : from.over_p(ld<BF16>(row_of<BF16>(a, at), v));
            lp = fma(x, 0.693147180559945309417, -log(sh.p[tid].s));
        }
        a.tokens[at] = (int32_t)v;
        a.logprob[at] = (float)lp;
    }
    if (tid == 0) a.count[b] = sh.count;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace verify

using namespace verify;

void verify_plan(VerifyArgs& a, bool bf16, bool drafted) {
    a.rows = (int64_t)a.batch * (a.drafts + 1 + (drafted ? a.drafts : 0));
    // Workgroups for 8 a CU, of at least 2048 values each.
    const int64_t round = kThreads * (bf16 ? 8 : 4);
    int64_t splits = (2048 + a.rows - 1) / a.rows;
    const int64_t most = (a.V + 2047) / 2048;
    if (splits > most) splits = most;
    if (splits > 64) splits = 64;
    a.per = ((a.V + splits - 1) / splits + round - 1) / round * round;
    a.splits = (int)((a.V + a.per - 1) / a.per);
    // Pieces of 2048 values for few sequences, where a workgroup's chain of trips to
    // memory counts, and up to 8192, where their number does.
    a.piece = 2048;
    while (a.piece < 8192 && a.batch * ((a.V + a.piece - 1) / a.piece) > 1024) a.piece *= 2;
    a.pieces = (int)((a.V + a.piece - 1) / a.piece);
}

VerifyWs verify_ws(const VerifyArgs& a) {
    VerifyWs w{};
    w.part = 0;
    w.mass = up256((size_t)a.rows * a.splits * 2 * sizeof(double));
    w.done = w.mass + up256((size_t)a.batch * a.pieces * 2 * sizeof(double));
    w.total = w.done + up256((size_t)a.batch * sizeof(uint32_t));
    return w;
}

int64_t verify_workgroups(const VerifyArgs& a) {
    const int64_t x = a.rows * a.splits, y = (int64_t)a.batch * a.pieces;
    return x > y ? x : y;
}

hipError_t launch_verify(VerifyArgs a, bool bf16, void* workspace, hipStream_t s) {
    const VerifyWs w = verify_ws(a);
    a.part = (double*)((char*)workspace + w.part);
    a.mass = (double*)((char*)workspace + w.mass);
    a.done = (uint32_t*)((char*)workspace + w.done);
    const unsigned n = (unsigned)(a.rows * a.splits), m = (unsigned)((int64_t)a.batch * a.pieces);
    {
        ProfScope ps(s, kPhaseMain);
        if (bf16) verify_sum_kernel<true><<<n, kThreads, 0, s>>>(a);
        else verify_sum_kernel<false><<<n, kThreads, 0, s>>>(a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ProfScope ps(s, kPhaseReduce);
    if (bf16) verify_draw_kernel<true><<<m, kThreads, 0, s>>>(a);
    else verify_draw_kernel<false><<<m, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace msscan
