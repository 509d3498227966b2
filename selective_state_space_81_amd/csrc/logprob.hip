// logprob.hip -- log probabilities of given tokens, with the entropy of each
// row and its most likely alternatives (ms_token_logprobs_fwd), and the
// gradient (ms_token_logprobs_bwd).  With x = scale * logit:
//
//   lse = log sum_v e^x_v,  logprob = x_t - lse,  H = lse - sum_v p_v x_v
//   dlogit_v = scale * (g_lp ([v = t] - p_v) - g_H p_v (log p_v + H))
//
// Both are bound by memory: the forward reads every logit once, the gradient
// reads and writes each once.  The forward keeps, per lane, a reference r near
// the running maximum, s = sum 2^d and T = sum d 2^d with d = c logit - r (one
// fused operation) and c = scale log2 e, moved to a new reference by
// (s, T) -> 2^delta (s, T + delta s).  Sums of d, not of x, so that the entropy
// ln2 (log2 s - T / s) has no cancellation against a large maximum.
//
// Alternatives come from the same pass.  A wave holds a threshold that at least
// `top` logits of the row reach: the top-th largest of the maxima of the
// workgroup's lanes (or of groups of lanes, Threshold below) over their first
// block.  A lane whose block of 16 (8 in fp32) logits reaches it, known from the
// maximum that the softmax needs anyway, notes the block (logprob_notes.h): one
// comparison a block, and some five notes in 4000 normal logits at top 5.  At the
// end the threshold is taken once more, from the maxima over all blocks, and few
// of the noted blocks reach it; those are read again (they are in cache), and
// each logit that reaches it finds its rank by counting the larger ones of the
// workgroup, in LDS.
//
// Measured (5.6 TB/s is what a copy reaches): 8192 x 50280 bf16 with 5
// alternatives 148 to 182 us (824 MB, 5.6 to 4.5 TB/s, as much of it as is still
// in the last-level cache); 8192 x 32001 bf16, none, 129 us, and its gradient 173
// (1.05 GB, 6.1 TB/s); 64 x 131072 bf16 with 20 alternatives 12.2 + 4.1 us and
// one row of 50280 fp32 9.6, both bound by latency: three trips to memory, five
// barriers and, in the first, a second launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "lm_internal.h"
#include "logprob_notes.h"
#include "msscan_internal.h"

namespace msscan {
namespace {

using namespace dev;

constexpr int kMaxKeys = 1024;  // keys that a workgroup ranks
// References stay within +-kFar; a row whose largest logit is past it (all of
// them the type's lowest value, say) has its sums taken again by far_row.
constexpr float kFar = 1e38f;
// Exponents below this give 2^d = 0 in fp32; d is held here in the products
// d 2^d, where -inf times 0 would be NaN.
constexpr float kDead = -200.f;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef u4 u4_align2 __attribute__((aligned(2)));
typedef u4 u4_align4 __attribute__((aligned(4)));

template <bool BF16>
struct Lg {
    static constexpr int N = BF16 ? 8 : 4;  // logits in 16 bytes
    typedef typename std::conditional<BF16, uint16_t, float>::type E;
    typedef u4 T;
    // rows are aligned to their element only
    typedef typename std::conditional<BF16, u4_align2, u4_align4>::type M;
    static __device__ __forceinline__ T load(const E* p) { return *reinterpret_cast<const M*>(p); }
    static __device__ __forceinline__ void unpack(T w, float (&v)[N]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (BF16) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            } else {
                v[k] = __uint_as_float(w[k]);
            }
        }
    }
    static __device__ __forceinline__ void store(E* p, const float (&v)[N]) {
        T w;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (BF16)
                w[k] = (uint32_t)f32_to_bf16_rne(v[2 * k]) |
                       ((uint32_t)f32_to_bf16_rne(v[2 * k + 1]) << 16);
            else
                w[k] = __float_as_uint(v[k]);
        }
        *reinterpret_cast<M*>(p) = w;
    }
    static __device__ __forceinline__ float one(const E* p) {
        if constexpr (BF16) return __uint_as_float((uint32_t)*p << 16);
        else return *p;
    }
};

__device__ __forceinline__ int64_t target_of(const LogprobArgs& a, int64_t row) {
    if (!a.targets) return -1;
    const int64_t t = a.wide ? static_cast<const int64_t*>(a.targets)[row]
                             : (int64_t) static_cast<const int32_t*>(a.targets)[row];
    return t < a.V ? t : -1;
}

// ---- reductions over a wave ------------------------------------------------------------
// Within 16 lanes through DPP (the four steps pair each lane with one that
// holds another part), then the four rows' values from the scalar side.
template <class F>
__device__ __forceinline__ float wave_reduce(float v, F f) {
    auto step = [&](auto ctrl) {
        v = f(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value,
                                                         0xf, 0xf, true)));
    };
    step(std::integral_constant<int, 0xB1>{});   // quad_perm 1,0,3,2
    step(std::integral_constant<int, 0x4E>{});   // quad_perm 2,3,0,1
    step(std::integral_constant<int, 0x141>{});  // row_half_mirror
    step(std::integral_constant<int, 0x140>{});  // row_mirror
    auto row = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
    return f(f(row(0), row(16)), f(row(32), row(48)));
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_reduce(v, [](float a, float b) { return a + b; });
}

// ---- softmax statistics ---------------------------------------------------------------
struct Stat {
    float r, s, T;
    __device__ __forceinline__ void move(float to) {
        const float dl = fmaxf(r - to, kDead), f = hw_exp2(dl);
        T = f * fmaf(dl, s, T);
        s *= f;
        r = to;
    }
    __device__ __forceinline__ void join_wave() {
        move(wave_max(r));
        s = wave_sum(s);
        T = wave_sum(T);
    }
};

// ---- alternatives -----------------------------------------------------------------------
// Order of a value as an unsigned number (-0 counts as 0), then lower tokens
// first.  0 is no entry.
__device__ __forceinline__ uint64_t top_key(float v, uint32_t token) {
    const uint32_t b = __float_as_uint(v + 0.f);
    const uint32_t o = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~token;
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}

// LDS between lanes of one wave: its accesses stay in order.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int l) {
    const uint32_t lo = __shfl((uint32_t)v, l), hi = __shfl((uint32_t)(v >> 32), l);
    return ((uint64_t)hi << 32) | lo;
}

// One compare-exchange of a bitonic network: lanes with `high` keep the larger.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int lane, int stride, bool high) {
    const uint64_t o = shfl64(v, lane ^ stride);
    return (v > o) == high ? v : o;
}

// The 64 largest of a sorted list and 64 values in any order, largest in lane 0.
__device__ __forceinline__ uint64_t merge_in(uint64_t list, uint64_t v, int lane) {
#pragma unroll 1
    for (int size = 2; size <= 64; size <<= 1)
#pragma unroll 1
        for (int stride = size >> 1; stride > 0; stride >>= 1)
            v = exchange(v, lane, stride, ((lane & stride) == 0) == ((lane & size) == 0));
    v = shfl64(v, 63 - lane);
    v = v > list ? v : list;
#pragma unroll 1
    for (int stride = 32; stride > 0; stride >>= 1)
        v = exchange(v, lane, stride, (lane & stride) == 0);
    return v;
}

// The wave that Noted runs on.
struct Wave {
    static __device__ __forceinline__ uint64_t ballot(bool v) { return __ballot(v); }
    static __device__ __forceinline__ void sync() { wave_sync(); }
};

// A value that at least `top` logits of the workgroup reach: the top-th largest
// of the maxima of its lanes, or of neighbouring lanes together, four maxima or
// more for each alternative (that is almost as high, and fewer are compared).
template <int W>
struct Threshold {
    float high[64 * W], least[W];

    // By the whole workgroup; two barriers.  lane_max: -inf where there is none.
    __device__ __forceinline__ float take(float lane_max, int top) {
        float v = lane_max == lane_max ? lane_max : -__builtin_inff();
        auto join = [&](auto ctrl) {
            v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(
                             __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true)));
        };
        // log2 of the lanes together, 4 at most (a DPP row)
        int shift = top <= 8 ? 3 : top <= 16 ? 2 : top <= 32 ? 1 : 0;
        if (W == 16) shift = min(shift + 2, 4);
        if (shift > 0) join(std::integral_constant<int, 0xB1>{});   // quad_perm 1,0,3,2
        if (shift > 1) join(std::integral_constant<int, 0x4E>{});   // quad_perm 2,3,0,1
        if (shift > 2) join(std::integral_constant<int, 0x141>{});  // row_half_mirror
        if (shift > 3) join(std::integral_constant<int, 0x140>{});  // row_mirror
        const int n = (64 * W) >> shift, tid = threadIdx.x;
        if ((tid & ((1 << shift) - 1)) == 0) high[tid >> shift] = v;
        __syncthreads();
        if ((tid & ~63) < n) {  // whole waves
            const float own = high[min(tid, n - 1)];
            int above = 0;
#pragma unroll 8
            for (int k = 0; k < n; k += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) above += high[k + e] > own;
            }
            const float lo = -wave_max(above < top ? -own : -__builtin_inff());
            if ((tid & 63) == 0) least[tid >> 6] = lo;
        }
        __syncthreads();
        float t = least[0];
        for (int w = 1; w * 64 < n; ++w) t = fminf(t, least[w]);
        return t;
    }
};

// The `top` best of n keys in LDS, sorted, to out[0 .. top) (0 where there are
// not so many): each key's rank is the number of larger ones.  A key that is
// not there is 0; others differ.  By the whole workgroup.
__device__ __forceinline__ void rank_keys(const uint64_t* key, int n, int top, uint64_t* out) {
    for (int k = threadIdx.x; k < top; k += blockDim.x) out[k] = 0;
    __syncthreads();
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
        const uint64_t v = key[k];
        int rank = 0;
#pragma unroll 8
        for (int q = 0; q < n; ++q) rank += key[q] > v;
        if (v && rank < top) out[rank] = v;
    }
    __syncthreads();
}

// What the rows' results are once the statistics and the sorted keys are
// known; high: the row's largest logit.
__device__ __forceinline__ void finish_row(const LogprobArgs& a, int64_t row, const Stat& st,
                                           float high, float target_logit, bool has_target,
                                           const uint64_t* best) {
    const float c = a.scale * kLog2e;
    const bool empty = high == -__builtin_inff() && st.s == 0.f;  // every logit is -inf
    const bool far = !(fabsf(high * c) < kFar);    // then r stands for high itself: see far_row
    const float l2 = empty ? 0.f : log2f(st.s);
    // Neither lse - scale * high nor the entropy is below 0; the rounding of r
    // can leave them there by 2^-24 of it (a NaN stays).
    auto at_least_0 = [](float v) { return v < 0.f ? 0.f : v; };
    const float rest = empty ? -__builtin_inff()
                             : at_least_0((l2 + (far ? 0.f : fmaf(-high, c, st.r))) * kLn2);
    // x - lse of a logit
    auto logp = [&](float v) {
        return empty ? -__builtin_inff() : fmaf(v - high, a.scale, -rest);
    };
    if (threadIdx.x == 0) {
        if (a.lse) a.lse[row] = empty ? rest : fmaf(high, a.scale, rest);
        if (a.stats) {
            a.stats[2 * row] = high;
            a.stats[2 * row + 1] = rest;
        }
        if (a.entropy) a.entropy[row] = empty ? 0.f : at_least_0(kLn2 * (l2 - st.T / st.s));
        if (a.logprob) a.logprob[row] = has_target ? logp(target_logit) : 0.f;
    }
    if ((int)threadIdx.x < a.top) {
        const uint64_t k = best[threadIdx.x];
        a.top_id[row * a.top + threadIdx.x] = k ? (int32_t)~(uint32_t)k : -1;
        a.top_logprob[row * a.top + threadIdx.x] = k ? logp(key_value(k)) : -__builtin_inff();
    }
}

// Joins the statistics of a few waves or splits, one a lane, in every lane
// ({r, s, T, largest logit} each, `stride` apart).
__device__ __forceinline__ Stat join_lanes(const float* part, int n, int stride, float& high) {
    const int lane = threadIdx.x & 63;
    Stat st{-kFar, 0.f, 0.f};
    float h = -__builtin_inff();
    if (lane < n) {
        const float* q = part + lane * stride;
        st = Stat{q[0], q[1], q[2]};
        h = q[3];
    }
    st.join_wave();
    high = wave_max(h);
    return st;
}

// s and T of a row whose largest logit is so far out that c * logit does not
// fit, with d = (logit - high) c, by one wave; r is left 0.
template <class L>
__device__ __forceinline__ Stat far_row(const typename L::E* x, int64_t V, float high, float c) {
    Stat st{0.f, 0.f, 0.f};
    for (int64_t i = threadIdx.x & 63; i < V; i += 64) {
        const float d = (L::one(x + i) - high) * c, w = hw_exp2(d);
        st.s += w;
        st.T = fmaf(w, fmaxf(d, kDead), st.T);
    }
    st.s = wave_sum(st.s);
    st.T = wave_sum(st.T);
    return st;
}

// The end of a row, by the workgroup's first wave, from parts as join_lanes reads them.
template <class L>
__device__ __forceinline__ void end_row(const LogprobArgs& a, int64_t row, const float* part, int n,
                                        const typename L::E* x, float target_logit,
                                        bool has_target, const uint64_t* best) {
    float high;
    Stat st = join_lanes(part, n, 4, high);
    const float c = a.scale * kLog2e;
    if (high != -__builtin_inff() && !(fabsf(high * c) < kFar)) st = far_row<L>(x, a.V, high, c);
    finish_row(a, row, st, high, target_logit, has_target, best);
}

// ---- forward ------------------------------------------------------------------------------
// One workgroup of W waves a row, or a split of one.  A wave takes blocks of 64 * U vectors
// in turn with the others, one in hand and D - 1 on the way.  Without
// alternatives (8192 x 32001 bf16): U, D = 4, 3 at 4 waves a SIMD 129 us; 4, 2 at
// 6 134; 2, 3 at 8 138; 1, 4 at 8 144.  With them registers hold U = 2 (U = 4, D =
// 2: 8192 x 50280 at 5 213 against 185).
template <bool BF16, bool TOP, int W>
__global__ void __launch_bounds__(64 * W, TOP && W == 4 ? 5 : 4) logprob_fwd(LogprobArgs a) {
    using L = Lg<BF16>;
    using E = typename L::E;
    constexpr int N = L::N, U = TOP ? 2 : 4;  // vectors a lane takes of a block
    constexpr int D = 3;                      // blocks in hand or under way
    __shared__ uint64_t s_key[TOP ? kMaxKeys : 1], s_best[TOP ? kMaxTop : 1];
    __shared__ Notes s_notes[TOP ? W : 1];
    __shared__ Threshold<W> s_level[1];
    __shared__ float s_stat[W][4], s_bound[W];
    __shared__ int s_count;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float c = a.scale * kLog2e;
    // the row, and this workgroup's vectors of it
    int64_t row = blockIdx.x;
    const uint32_t nvec = (uint32_t)(a.V / N);
    uint32_t v0 = 0, v1 = nvec;
    bool last = true;
    if (a.splits > 1) {
        const uint32_t split = blockIdx.x % (uint32_t)a.splits;
        row = blockIdx.x / (uint32_t)a.splits;
        v0 = min(split * a.per, nvec);
        v1 = min(v0 + a.per, nvec);
        last = split == (uint32_t)a.splits - 1;
    }
    const E* x = static_cast<const E*>(a.logits) + row * a.ld;

    Stat st{-kFar, 0.f, 0.f};
    float high = -__builtin_inff();  // the lane's largest logit
    Noted<Wave> noted;
    if constexpr (TOP) {
        noted.init(&s_notes[wave], a.top, lane);
        if (threadIdx.x == 0) s_count = 0;
    }

    // the lane's K logits (-inf where there is none; any: one is), from `token`
    auto take = [&](auto& v, auto K, bool any, uint32_t token) {
        constexpr int kN = decltype(K)::value;
        float mb = v[0];
#pragma unroll
        for (int e = 1; e < kN; ++e) mb = fmaxf(mb, v[e]);
        if constexpr (TOP) {
            const bool in = any && mb >= noted.thr;
            if (__any(in)) noted.note(in, token, mb);
        }
        high = fmaxf(high, mb);
        st.move(fminf(fmaxf(st.r, mb * c), kFar));
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float d = fmaf(v[e], c, -st.r), w = hw_exp2(d);
            st.s += w;
            st.T = fmaf(w, fmaxf(d, kDead), st.T);
        }
    };

    typename L::T w[D][U];
    auto load = [&](uint32_t b, typename L::T(&r)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = L::load(x + (int64_t)min(b + u * 64 + lane, v1 - 1) * N);
    };
    // a block's logits in order of their tokens; false where the lane has none
    auto unpack = [&](uint32_t b, const typename L::T(&r)[U], float(&v)[U * N]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float t[N];
            L::unpack(r[u], t);
#pragma unroll
            for (int e = 0; e < N; ++e) v[u * N + e] = t[e];
        }
        if (b + 64 * U <= v1) return true;
#pragma unroll
        for (int u = 0; u < U; ++u) {  // the end of the vectors
            const bool in = b + u * 64 + lane < v1;
#pragma unroll
            for (int e = 0; e < N; ++e) v[u * N + e] = in ? v[u * N + e] : -__builtin_inff();
        }
        return b + lane < v1;
    };
    auto block = [&](uint32_t b, const typename L::T(&r)[U]) {
        float v[U * N];
        const bool any = unpack(b, r, v);
        take(v, std::integral_constant<int, U * N>{}, any, (b + lane) * N);
    };
    constexpr uint32_t kStep = 64 * U * W;
    uint32_t b = v0 + wave * (64 * U);
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
        if (b + d * kStep < v1) load(b + d * kStep, w[d]);
    // the target's logit travels beside the row
    const int64_t target = target_of(a, row);
    float tl = 0.f;
    if (wave == 0 && target >= 0) tl = L::one(x + target);
    if constexpr (TOP) {
        float m = -__builtin_inff();
        if (b < v1) {
            float v[U * N];
            unpack(b, w[0], v);
            m = v[0];
#pragma unroll
            for (int e = 1; e < U * N; ++e) m = fmaxf(m, v[e]);
        }
        noted.thr = noted.bound = s_level[0].take(m, a.top);
    }
    // D - 1 blocks are under way while one is taken.  One body for all: three in
    // turn, without the moves, measured 10.3 against 9.7 us for a row of 50280
    // fp32 and 171 against 165 for 8192 of bf16, at top 5.
#pragma unroll 1
    for (; b < v1; b += kStep) {
        const uint32_t ahead = b + (D - 1) * kStep;
        if (ahead < v1) load(ahead, w[D - 1]);
        block(b, w[0]);
#pragma unroll
        for (int d = 0; d + 1 < D; ++d)
#pragma unroll
            for (int u = 0; u < U; ++u) w[d][u] = w[d + 1][u];
    }
    if (wave == 0 && last && (int64_t)nvec * N < a.V) {  // the row's last V % N logits
        const int64_t i = (int64_t)nvec * N + lane;
        const bool in = i < a.V;
        float v[1] = {in ? L::one(x + i) : -__builtin_inff()};
        take(v, std::integral_constant<int, 1>{}, in, (uint32_t)i);
    }
    float level = 0.f;
    if constexpr (TOP) {
        if (lane == 0) s_bound[wave] = noted.bound;
        level = s_level[0].take(high, a.top);
    }
    st.join_wave();
    high = wave_max(high);
    if (lane == 0) {
        s_stat[wave][0] = st.r;
        s_stat[wave][1] = st.s;
        s_stat[wave][2] = st.T;
        s_stat[wave][3] = high;
    }
    __syncthreads();
    const int64_t at = row * a.splits + (a.splits > 1 ? blockIdx.x % (uint32_t)a.splits : 0);
    if constexpr (TOP) {
        // Noted blocks that reach the row's last threshold, G logits each, read
        // again 64 / G blocks at a time; f gets every logit that reaches it.
        float t = level;
#pragma unroll
        for (int k = 0; k < W; ++k) t = fmaxf(t, s_bound[k]);
        constexpr int G = U * N;
        auto read_again = [&](auto f) {
            const Notes& q = s_notes[wave];
            for (int k0 = 0; k0 < noted.count; k0 += 64) {
                const bool in = k0 + lane < noted.count && q.high[k0 + lane] >= t;
                uint64_t m = __ballot(in);
                const uint32_t mine = in ? q.first[k0 + lane] : 0;
                while (m) {
                    uint32_t from = 0xffffffffu;
#pragma unroll
                    for (int g = 0; g < 64 / G; ++g) {
                        if (!m) break;
                        const int l = __ffsll((unsigned long long)m) - 1;
                        m &= m - 1;
                        const uint32_t v = __builtin_amdgcn_readlane(mine, l);
                        if (lane / G == g) from = v;
                    }
                    const int e = lane % G;
                    const uint32_t tok = from + e / N * (64 * N) + e % N;
                    // a block ends with the vectors; the logits after them are alone
                    const bool have = from != 0xffffffffu &&
                                      (from < v1 * N ? tok < v1 * N : e == 0 && tok < (uint32_t)a.V);
                    float v = -__builtin_inff();
                    if (have) v = L::one(x + tok);
                    f(have && v >= t, v, tok);
                }
            }
        };
        read_again([&](bool in, float v, uint32_t tok) {
            if (!in) return;
            const int at = atomicAdd(&s_count, 1);  // any order: ranks do not depend on it
            if (at < kMaxKeys) s_key[at] = top_key(v, tok);
        });
        __syncthreads();
        int n = s_count;
        if (n > kMaxKeys) {  // many equal logits: each wave's 64 best by merging
            uint64_t list = 0;
            read_again([&](bool in, float v, uint32_t tok) {
                list = merge_in(list, in ? top_key(v, tok) : 0, lane);
            });
            __syncthreads();
            s_key[wave * 64 + lane] = list;
            n = 64 * W;
            __syncthreads();
        }
        rank_keys(s_key, n, a.top, s_best);
    }
    if (a.splits > 1) {
        if constexpr (TOP) {
            if ((int)threadIdx.x < a.top) a.list[at * a.top + threadIdx.x] = s_best[threadIdx.x];
        }
        if (wave != 0) return;
        st = join_lanes(&s_stat[0][0], W, 4, high);
        if (lane == 0) {
            a.part[at * 4] = st.r;
            a.part[at * 4 + 1] = st.s;
            a.part[at * 4 + 2] = st.T;
            a.part[at * 4 + 3] = high;
        }
        return;
    }
    if (wave != 0) return;
    end_row<L>(a, row, &s_stat[0][0], W, x, tl, target >= 0, s_best);
}

// Joins the splits of a row (64 at most, and kMaxKeys keys).
constexpr int kJoinWaves = 4;
template <bool BF16, bool TOP>
__global__ void __launch_bounds__(64 * kJoinWaves) logprob_join(LogprobArgs a) {
    using L = Lg<BF16>;
    __shared__ uint64_t s_key[TOP ? kMaxKeys : 1], s_best[TOP ? kMaxTop : 1];
    const int64_t row = blockIdx.x;
    const typename L::E* x = static_cast<const typename L::E*>(a.logits) + row * a.ld;
    const int64_t target = target_of(a, row);
    float tl = 0.f;
    if (threadIdx.x == 0 && target >= 0) tl = L::one(x + target);
    if constexpr (TOP) {
        // A key that at least `top` keys reach: each split's j-th is reached by
        // j of its own, so the k-th largest of those, k j >= top.  Few reach it.
        __shared__ uint64_t s_bound, s_jth[64];
        __shared__ int s_count;
        const uint64_t* list = a.list + row * a.splits * a.top;
        const int j = (a.top + a.splits - 1) / a.splits, kth = (a.top + j - 1) / j;
        const uint64_t own = (int)threadIdx.x < a.splits ? list[threadIdx.x * a.top + j - 1] : 0;
        if (threadIdx.x < 64) s_jth[threadIdx.x] = own;
        if (threadIdx.x == 0) s_bound = 0, s_count = 0;
        __syncthreads();
        if ((int)threadIdx.x < a.splits && own) {  // keys differ: one rank is kth - 1
            int above = 0;
            for (int q = 0; q < a.splits; ++q) above += s_jth[q] > own;
            if (above == kth - 1) s_bound = own;
        }
        __syncthreads();
        for (int k = threadIdx.x; k < a.splits * a.top; k += 64 * kJoinWaves) {
            const uint64_t v = list[k];
            if (v && v >= s_bound) s_key[atomicAdd(&s_count, 1)] = v;
        }
        __syncthreads();
        rank_keys(s_key, s_count, a.top, s_best);
    }
    if (threadIdx.x >= 64) return;
    end_row<L>(a, row, a.part + row * a.splits * 4, a.splits, x, tl, target >= 0, s_best);
}

// ---- gradient -------------------------------------------------------------------------------
// Vectors a thread takes (8192 x 32001 bf16, 1.05 GB: 173 us, 6.1 TB/s; with 1 211,
// with 4 or 8 182, with non-temporal stores 182).
constexpr int kGradVecs = 2;

template <bool BF16>
__global__ void __launch_bounds__(256) logprob_bwd(LogprobArgs a, uint32_t chunks) {
    using L = Lg<BF16>;
    using E = typename L::E;
    constexpr int N = L::N;
    const int64_t row = (int64_t)(blockIdx.x / chunks);
    const int64_t first = (int64_t)(blockIdx.x % chunks) * (256 * kGradVecs);
    const E* x = static_cast<const E*>(a.logits) + row * a.ld;
    E* o = static_cast<E*>(a.dlogits) + row * a.ldd;
    const float m = a.stats[2 * row], lns = a.stats[2 * row + 1];
    const bool empty = lns == -__builtin_inff();  // nothing left by the mask: no gradient
    const int64_t target = target_of(a, row);
    const float gl = (a.dlogprob && target >= 0 ? a.dlogprob[row] : 0.f) * a.scale;
    const float gh = (a.dentropy ? a.dentropy[row] : 0.f) * a.scale;
    const float ent = a.entropy ? a.entropy[row] : 0.f;
    // -p (gl + gh H + gh log p)
    const float g0 = fmaf(gh, ent, gl);
    auto grad = [&](float v) {
        const float lp = fmaf(v - m, a.scale, -lns);
        const float p = hw_exp2(lp * kLog2e);
        const float g = -p * fmaf(gh, lp, g0);
        return empty || p == 0.f ? 0.f : g;  // 0 times a huge log p is 0
    };
    const int64_t nvec = a.V / N, tv = target >= 0 ? target / N : -1;
    typename L::T w[kGradVecs];
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
        const int64_t i = first + u * 256 + threadIdx.x;
        if (i < nvec) w[u] = L::load(x + i * N);
    }
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
        const int64_t i = first + u * 256 + threadIdx.x;
        if (i >= nvec) continue;
        float v[N];
        L::unpack(w[u], v);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = grad(v[e]);
        if (i == tv && !empty) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e == (int)(target - tv * N)) v[e] += gl;
        }
        L::store(o + i * N, v);
    }
    const int64_t i = nvec * N + threadIdx.x;
    if (first + 256 * kGradVecs >= nvec && i < a.V) {
        float v = grad(L::one(x + i));
        if (i == target && !empty) v += gl;
        if constexpr (BF16) o[i] = f32_to_bf16_rne(v);
        else o[i] = v;
    }
}

uint32_t grad_chunks(const LogprobArgs& a, bool bf16) {
    const int64_t nvec = a.V / (bf16 ? 8 : 4);
    const int64_t n = (nvec + 256 * kGradVecs - 1) / (256 * kGradVecs);
    return (uint32_t)(n < 1 ? 1 : n);
}

}  // namespace

void logprob_plan(LogprobArgs& a, bool bf16) {
    // Few rows are split over about 512 workgroups, of 4096 logits at least (64
    // rows of 131072 at top 20: 17.0 us, with 1024 18.5).
    const int64_t vec = bf16 ? 8 : 4, nvec = a.V / vec;
    int64_t n = a.rows > 0 ? (512 + a.rows - 1) / a.rows : 1;
    const int64_t most = (a.V + 4095) / 4096, keys = a.top ? kMaxKeys / a.top : 64;
    if (n > most) n = most;
    if (n > keys) n = keys;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    // Instead of splits, one workgroup of 16 waves a row, with no second launch:
    // for rows that are short, or fill the chip (256 of them: a compute unit
    // each), as GPU time alone at top 5 has it, in us split and whole: one row of
    // 20000 bf16 8.8 and 7.4, of 50280 fp32 9.6 and 10.5 (and 2 between the
    // launches), of 131072 bf16 9.1 and 13.9; 64 of those 13.2 and 15.5, 96 16.9
    // and 15.9, 200 21.7 and 18.0, 260 25.8 and 30.8.
    const int64_t bytes = a.V * (bf16 ? 2 : 4);
    a.waves = 4;
    if (n > 1 && a.rows <= 256 && (a.rows >= 96 || bytes <= 224 * 1024)) a.waves = 16, n = 1;
    const int64_t per = (nvec + n - 1) / n;
    a.per = (uint32_t)((per + 63) / 64 * 64);  // whole waves of vectors
    a.splits = n == 1 ? 1 : (int)((nvec + a.per - 1) / a.per);
    if (a.splits < 1) a.splits = 1;
}

LogprobWs logprob_ws(const LogprobArgs& a) {
    LogprobWs w{};
    if (a.splits < 2) return w;
    const size_t n = (size_t)a.rows * (size_t)a.splits;
    w.part = 0;
    w.list = (n * 16 + 255) / 256 * 256;
    w.total = w.list + n * (size_t)a.top * 8;
    return w;
}

template <int W>
static void fwd_variant(const LogprobArgs& a, bool bf16, hipStream_t s) {
    const dim3 grid((unsigned)(a.rows * a.splits)), blk(64 * W);
    if (bf16) {
        if (a.top) hipLaunchKernelGGL((logprob_fwd<true, true, W>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((logprob_fwd<true, false, W>), grid, blk, 0, s, a);
    } else {
        if (a.top) hipLaunchKernelGGL((logprob_fwd<false, true, W>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((logprob_fwd<false, false, W>), grid, blk, 0, s, a);
    }
}

hipError_t launch_logprob_fwd(LogprobArgs a, bool bf16, void* workspace, hipStream_t s) {
    const LogprobWs w = logprob_ws(a);
    if (a.splits > 1) {
        a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.part);
        a.list = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + w.list);
    }
    {
        ProfScope ps(s, kPhaseMain);
        if (a.waves == 16) fwd_variant<16>(a, bf16, s);
        else fwd_variant<4>(a, bf16, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    ProfScope ps(s, kPhaseReduce);
    const dim3 rows((unsigned)a.rows), blk(64 * kJoinWaves);
    if (bf16) {
        if (a.top) hipLaunchKernelGGL((logprob_join<true, true>), rows, blk, 0, s, a);
        else hipLaunchKernelGGL((logprob_join<true, false>), rows, blk, 0, s, a);
    } else {
        if (a.top) hipLaunchKernelGGL((logprob_join<false, true>), rows, blk, 0, s, a);
        else hipLaunchKernelGGL((logprob_join<false, false>), rows, blk, 0, s, a);
    }
    return hipGetLastError();
}

int64_t logprob_bwd_workgroups(const LogprobArgs& a, bool bf16) {
    return a.rows * (int64_t)grad_chunks(a, bf16);
}

hipError_t launch_logprob_bwd(const LogprobArgs& a, bool bf16, hipStream_t s) {
    ProfScope ps(s, kPhaseMain);
    const uint32_t chunks = grad_chunks(a, bf16);
    const dim3 grid((unsigned)(a.rows * chunks)), blk(256);
    if (bf16) hipLaunchKernelGGL((logprob_bwd<true>), grid, blk, 0, s, a, chunks);
    else hipLaunchKernelGGL((logprob_bwd<false>), grid, blk, 0, s, a, chunks);
    return hipGetLastError();
}

}  // namespace msscan
