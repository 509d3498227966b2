// logprob.hip -- log probabilities of given tokens, with the entropy of each
// row and its most likely alternatives (ms_token_logprobs_fwd), and the
// gradient (ms_token_logprobs_bwd).  With x = scale * logit:
//
//   lse = log sum_v e^x_v,  logprob = x_t - lse,  H = lse - sum_v p_v x_v
//   dlogit_v = scale * (g_lp ([v = t] - p_v) - g_H p_v (log p_v + H))
//
// Both are bound by memory: the forward reads every logit once, the gradient
// reads and writes each once.  The forward keeps, per lane, the running
// maximum m, s = sum 2^d and T = sum d 2^d with d = (logit - m) c and
// c = scale log2 e, moved to a new maximum by (s, T) -> 2^delta (s, T + delta s).
// Sums of d, not of x, so that the entropy ln s - ln2 T / s has no
// cancellation against a large maximum.
//
// Alternatives come from the same pass.  A wave holds a threshold that at least
// `top` of its logits reach, first from the maxima of its lanes' first block
// (the top-th largest of 64), and notes the tokens that reach it; blocks whose
// maximum, known from the softmax, stays below cost one comparison.  Few tokens
// are noted (some ten of 10000 at top 5), so at the end each finds its rank by
// counting the larger ones of its workgroup, in LDS.  Should more than 64 come
// together before that (rows that rise), the wave sorts them, keeps the best
// and raises its threshold.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "lm_internal.h"
#include "msscan_internal.h"

namespace msscan {
namespace {

using namespace dev;

#ifndef LP_OCC
#define LP_OCC 4
#endif
#ifndef LP_WG
#define LP_WG 1024
#endif
#ifndef LP_MIN
#define LP_MIN 4096
#endif
constexpr int kLpWaves = 4;
constexpr int kMaxJoin = 1024;  // keys of a row's splits together
constexpr float kLowest = -3.402823466e38f;
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
    float m, s, T;
    __device__ __forceinline__ void move(float mn, float c) {
        const float dl = fmaxf((m - mn) * c, kDead), f = hw_exp2(dl);
        T = f * fmaf(dl, s, T);
        s *= f;
        m = mn;
    }
    __device__ __forceinline__ void join_wave(float c) {
        move(wave_max(m), c);
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

// The smallest float above v (x > v is then x >= next for every fp32 x).
__device__ __forceinline__ float next_above(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return __uint_as_float((b >> 31) ? b - 1 : b + 1);
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

// What a wave has noted: up to 127 tokens in LDS (its own part), and, once
// more than 64 have come together, the best of those before them as a list.
template <class L>
struct Noted {
    const typename L::E* x;  // the row
    uint32_t* tok;           // [128]
    uint64_t list;           // lane l: the (l+1)-th best so far, or 0
    float thr;               // what a logit has to reach to be noted
    int top, count, lane;
    bool listed;

    __device__ __forceinline__ void init(const typename L::E* row, uint32_t* t, int top_,
                                         int lane_) {
        x = row;
        tok = t;
        list = 0;
        thr = -__builtin_inff();
        top = top_;
        count = 0;
        lane = lane_;
        listed = false;
    }
    // First threshold: the top-th largest lane maximum, as the least of those
    // with fewer than `top` above them.
    __device__ __forceinline__ void seed(float lane_max) {
        const float v = lane_max == lane_max ? lane_max : -__builtin_inff();
        int above = 0;
#pragma unroll 16
        for (int l = 0; l < 64; ++l)
            above += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)) > v;
        thr = -wave_max(above < top ? -v : -__builtin_inff());
    }
    __device__ __forceinline__ uint64_t key_at(int k) const {
        const uint32_t t = tok[k];
        return top_key(L::one(x + t), t);
    }
    // Logits of later blocks have higher tokens than those of the list, so a
    // tie with the top-th does not enter.
    __device__ __forceinline__ void flush() {
        wave_sync();
        const uint64_t v = lane < count ? key_at(lane) : 0;
        const uint32_t rest = lane + 64 < count ? tok[lane + 64] : 0;
        wave_sync();
        tok[lane] = rest;
        count = count > 64 ? count - 64 : 0;
        list = merge_in(list, v, lane);
        listed = true;
        const uint64_t k = shfl64(list, top - 1);
        if (k) thr = next_above(key_value(k));
    }
    // Notes the lane's tokens first + (bit / N) * 64 N + bit % N, one for each
    // bit of `bits`.
    template <int N>
    __device__ __forceinline__ void note(uint32_t bits, uint32_t first) {
        for (;;) {
            const uint64_t m = __ballot(bits != 0);
            if (!m) return;
            if (bits) {
                const int b = __builtin_ctz(bits);
                bits &= bits - 1;
                tok[count + __popcll(m & ((1ull << lane) - 1))] = first + b / N * (64 * N) + b % N;
            }
            count += __popcll(m);
            if (count >= 64) flush();
        }
    }
};

// The `top` best of n keys in LDS, sorted, to out[0 .. top) (0 where there are
// not so many): each key's rank is the number of larger ones.  A key that is
// not there is 0; others differ.
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

// What the rows' results are once the statistics and the sorted keys are known.
__device__ __forceinline__ void finish_row(const LogprobArgs& a, int64_t row, const Stat& st,
                                           float target_logit, bool has_target,
                                           const uint64_t* best) {
    const bool empty = st.s == 0.f;  // every logit is -inf
    const float lns = empty ? 0.f : logf(st.s);
    if (threadIdx.x == 0) {
        if (a.lse) a.lse[row] = empty ? -__builtin_inff() : fmaf(st.m, a.scale, lns);
        if (a.stats) {
            a.stats[2 * row] = st.m;
            a.stats[2 * row + 1] = empty ? -__builtin_inff() : lns;
        }
        if (a.entropy) a.entropy[row] = empty ? 0.f : lns - kLn2 * (st.T / st.s);
        if (a.logprob) {
            float lp = 0.f;
            if (has_target)
                lp = empty ? -__builtin_inff() : (target_logit - st.m) * a.scale - lns;
            a.logprob[row] = lp;
        }
    }
    if ((int)threadIdx.x < a.top) {
        const uint64_t k = best[threadIdx.x];
        float lp = -__builtin_inff();
        if (k && !empty) lp = (key_value(k) - st.m) * a.scale - lns;
        a.top_id[row * a.top + threadIdx.x] = k ? (int32_t)~(uint32_t)k : -1;
        a.top_logprob[row * a.top + threadIdx.x] = lp;
    }
}

// Joins the statistics of a few waves or splits, one a lane, in every lane.
__device__ __forceinline__ Stat join_lanes(const float* part, int n, int stride, float c) {
    const int lane = threadIdx.x & 63;
    Stat st{kLowest, 0.f, 0.f};
    if (lane < n) st = Stat{part[lane * stride], part[lane * stride + 1], part[lane * stride + 2]};
    st.join_wave(c);
    return st;
}

// ---- forward ------------------------------------------------------------------------------
template <bool BF16, bool TOP>
__global__ void __launch_bounds__(64 * kLpWaves, LP_OCC) logprob_fwd(LogprobArgs a) {
    using L = Lg<BF16>;
    using E = typename L::E;
    constexpr int N = L::N, U = 4;  // vectors a lane takes of a block
    __shared__ uint64_t s_key[TOP ? kLpWaves * 128 : 1], s_best[TOP ? kMaxTop : 1];
    __shared__ uint32_t s_tok[TOP ? kLpWaves : 1][TOP ? 128 : 1];
    __shared__ float s_stat[kLpWaves][3];
    __shared__ int s_count[kLpWaves];
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

    Stat st{kLowest, 0.f, 0.f};
    Noted<L> noted;
    if constexpr (TOP) noted.init(x, s_tok[wave], a.top, lane);
    bool first = true;

    // the lane's K logits (-inf where there is none: `have` of them are)
    auto take = [&](auto& v, auto K, uint32_t have, uint32_t token) {
        constexpr int kN = decltype(K)::value;
        float mb = v[0];
#pragma unroll
        for (int e = 1; e < kN; ++e) mb = fmaxf(mb, v[e]);
        if constexpr (TOP) {
            if (first) {
                noted.seed(mb);
                first = false;
            }
            if (__any(mb >= noted.thr)) {
                uint32_t bits = 0;
#pragma unroll
                for (int e = kN - 1; e >= 0; --e) bits = 2 * bits + (v[e] >= noted.thr ? 1u : 0u);
                noted.template note<N>(bits & have, token);
            }
        }
        st.move(fmaxf(st.m, mb), c);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float d = (v[e] - st.m) * c, w = hw_exp2(d);
            st.s += w;
            st.T = fmaf(w, fmaxf(d, kDead), st.T);
        }
    };

    typename L::T w[U], nx[U];
    auto load = [&](uint32_t b, typename L::T(&r)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = L::load(x + (int64_t)min(b + u * 64 + lane, v1 - 1) * N);
    };
    uint32_t b = v0 + wave * (64 * U);
    if (b < v1) load(b, w);
    // the target's logit travels beside the row
    const int64_t target = target_of(a, row);
    float tl = 0.f;
    if (wave == 0 && target >= 0) tl = L::one(x + target);
    for (; b < v1; b += 64 * U * kLpWaves) {
        const uint32_t bn = b + 64 * U * kLpWaves;
        if (bn < v1) load(bn, nx);
        float v[U * N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float t[N];
            L::unpack(w[u], t);
#pragma unroll
            for (int e = 0; e < N; ++e) v[u * N + e] = t[e];
        }
        uint32_t have = U * N == 32 ? 0xffffffffu : (1u << (U * N)) - 1;
        if (b + 64 * U > v1) {  // the end of the vectors
            have = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = b + u * 64 + lane < v1;
                if (in) have |= ((1u << N) - 1) << (u * N);
#pragma unroll
                for (int e = 0; e < N; ++e) v[u * N + e] = in ? v[u * N + e] : -__builtin_inff();
            }
        }
        take(v, std::integral_constant<int, U * N>{}, have, (b + lane) * N);
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = nx[u];
    }
    if (wave == 0 && last && (int64_t)nvec * N < a.V) {  // the row's last V % N logits
        const int64_t i = (int64_t)nvec * N + lane;
        const bool in = i < a.V;
        float v[1] = {in ? L::one(x + i) : -__builtin_inff()};
        take(v, std::integral_constant<int, 1>{}, in ? 1u : 0u, (uint32_t)i);
    }
    st.join_wave(c);
    if (lane == 0) s_stat[wave][0] = st.m, s_stat[wave][1] = st.s, s_stat[wave][2] = st.T;
    const int64_t at = row * a.splits + (a.splits > 1 ? blockIdx.x % (uint32_t)a.splits : 0);
    if constexpr (TOP) {
        wave_sync();
        if (lane == 0) s_count[wave] = noted.count + (noted.listed ? a.top : 0);
        __syncthreads();
        int k0 = 0, n = 0;
#pragma unroll
        for (int k = 0; k < kLpWaves; ++k) {
            if (k == wave) k0 = n;
            n += s_count[k];
        }
        if (lane < noted.count) s_key[k0 + lane] = noted.key_at(lane);
        if (noted.listed && lane < a.top) s_key[k0 + noted.count + lane] = noted.list;
        __syncthreads();
        rank_keys(s_key, n, a.top, s_best);
    } else {
        __syncthreads();
    }
    if (a.splits > 1) {
        if constexpr (TOP) {
            if ((int)threadIdx.x < a.top) a.list[at * a.top + threadIdx.x] = s_best[threadIdx.x];
        }
        if (wave != 0) return;
        st = join_lanes(&s_stat[0][0], kLpWaves, 3, c);
        if (lane == 0) {
            a.part[at * 4] = st.m;
            a.part[at * 4 + 1] = st.s;
            a.part[at * 4 + 2] = st.T;
        }
        return;
    }
    if (wave != 0) return;
    st = join_lanes(&s_stat[0][0], kLpWaves, 3, c);
    finish_row(a, row, st, tl, target >= 0, s_best);
}

// Joins the splits of a row (64 at most, and kMaxJoin keys).
template <bool BF16, bool TOP>
__global__ void __launch_bounds__(64 * kLpWaves) logprob_join(LogprobArgs a) {
    using L = Lg<BF16>;
    __shared__ uint64_t s_key[TOP ? kMaxJoin : 1], s_best[TOP ? kMaxTop : 1];
    const int64_t row = blockIdx.x;
    const int64_t target = target_of(a, row);
    float tl = 0.f;
    if (threadIdx.x == 0 && target >= 0)
        tl = L::one(static_cast<const typename L::E*>(a.logits) + row * a.ld + target);
    if constexpr (TOP) {
        const int n = a.splits * a.top;
        for (int k = threadIdx.x; k < n; k += 64 * kLpWaves) s_key[k] = a.list[row * n + k];
        __syncthreads();
        rank_keys(s_key, n, a.top, s_best);
    }
    if (threadIdx.x >= 64) return;
    finish_row(a, row, join_lanes(a.part + row * a.splits * 4, a.splits, 4, a.scale * kLog2e), tl,
               target >= 0, s_best);
}

// ---- gradient -------------------------------------------------------------------------------
constexpr int kGradVecs = 4;  // vectors a thread takes

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
    // about 1024 workgroups, of LP_MIN logits at least
    const int64_t vec = bf16 ? 8 : 4, nvec = a.V / vec;
    int64_t n = a.rows > 0 ? (LP_WG + a.rows - 1) / a.rows : 1;
    const int64_t most = (a.V + LP_MIN - 1) / LP_MIN, keys = a.top ? kMaxJoin / a.top : 64;
    if (n > most) n = most;
    if (n > keys) n = keys;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
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

hipError_t launch_logprob_fwd(LogprobArgs a, bool bf16, void* workspace, hipStream_t s) {
    const LogprobWs w = logprob_ws(a);
    if (a.splits > 1) {
        a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.part);
        a.list = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + w.list);
    }
    const dim3 grid((unsigned)(a.rows * a.splits)), rows((unsigned)a.rows), blk(64 * kLpWaves);
    {
        ProfScope ps(s, kPhaseMain);
        if (bf16) {
            if (a.top) hipLaunchKernelGGL((logprob_fwd<true, true>), grid, blk, 0, s, a);
            else hipLaunchKernelGGL((logprob_fwd<true, false>), grid, blk, 0, s, a);
        } else {
            if (a.top) hipLaunchKernelGGL((logprob_fwd<false, true>), grid, blk, 0, s, a);
            else hipLaunchKernelGGL((logprob_fwd<false, false>), grid, blk, 0, s, a);
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    ProfScope ps(s, kPhaseReduce);
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
