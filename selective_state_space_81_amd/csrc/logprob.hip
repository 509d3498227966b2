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
// Alternatives come from the same pass.  A wave keeps its 64 best so far, one
// a lane, sorted by (value, lower token first) as one 64-bit key.  A block of
// logits is looked at closer only if some lane's maximum (known from the
// softmax) reaches the wave's current top-th value; the few that do are
// gathered in LDS and merged 64 at a time by a bitonic network.  The first
// threshold is the top-th largest of the lanes' own maxima, so that the start
// of the row does not pass whole.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "lm_internal.h"
#include "msscan_internal.h"

namespace msscan {
namespace {

using namespace dev;

constexpr int kLpWaves = 4;
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

// ---- softmax statistics ---------------------------------------------------------------
struct Stat {
    float m, s, T;
    __device__ __forceinline__ void move(float mn, float c) {
        const float dl = fmaxf((m - mn) * c, kDead), f = hw_exp2(dl);
        T = f * fmaf(dl, s, T);
        s *= f;
        m = mn;
    }
    __device__ __forceinline__ void join(float m2, float s2, float T2, float c) {
        Stat o{m2, s2, T2};
        const float mn = fmaxf(m, m2);
        move(mn, c);
        o.move(mn, c);
        s += o.s;
        T += o.T;
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

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m) {
    const uint32_t lo = __shfl_xor((uint32_t)v, m), hi = __shfl_xor((uint32_t)(v >> 32), m);
    return ((uint64_t)hi << 32) | lo;
}

// One compare-exchange of a bitonic network: lanes with `high` keep the larger.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int stride, bool high) {
    const uint64_t o = shfl_xor64(v, stride);
    return (v > o) == high ? v : o;
}

// The wave's 64 values, largest in lane 0.
__device__ __forceinline__ uint64_t sort64(uint64_t v, int lane) {
#pragma unroll
    for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1)
            v = exchange(v, stride, ((lane & stride) == 0) == ((lane & size) == 0));
    return v;
}

// The 64 largest of two sorted lists, sorted.
__device__ __forceinline__ uint64_t merge64(uint64_t a, uint64_t b, int lane) {
    const uint32_t lo = __shfl((uint32_t)b, 63 - lane), hi = __shfl((uint32_t)(b >> 32), 63 - lane);
    const uint64_t r = ((uint64_t)hi << 32) | lo;
    uint64_t v = a > r ? a : r;
#pragma unroll
    for (int stride = 32; stride > 0; stride >>= 1) v = exchange(v, stride, (lane & stride) == 0);
    return v;
}

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
    return ((uint64_t)hi << 32) | lo;
}

// The smallest float above v (v > x is then x' >= next for every fp32 x').
__device__ __forceinline__ float next_above(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return __uint_as_float((b >> 31) ? b - 1 : b + 1);
}

// LDS between lanes of one wave: its accesses stay in order.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct WaveTop {
    uint64_t list;  // lane l: the (l+1)-th best so far, or 0
    float thr;      // what a logit has to reach to be gathered
    int top, count, lane;
    uint64_t* buf;  // [128] in LDS, the wave's own

    __device__ __forceinline__ void init(int top_, int lane_, uint64_t* b) {
        list = 0;
        thr = -__builtin_inff();
        top = top_;
        count = 0;
        lane = lane_;
        buf = b;
    }
    // Logits of later blocks have higher tokens than those of the list, so a
    // tie with the top-th does not enter.
    __device__ __forceinline__ void set_threshold() {
        const uint64_t k = lane_value(list, top - 1);
        thr = k ? next_above(key_value(k)) : -__builtin_inff();
    }
    __device__ __forceinline__ void flush() {
        wave_sync();
        uint64_t v = lane < count ? buf[lane] : 0;
        const uint64_t rest = lane + 64 < count ? buf[lane + 64] : 0;
        wave_sync();
        buf[lane] = rest;
        wave_sync();
        count = count > 64 ? count - 64 : 0;
        list = merge64(list, sort64(v, lane), lane);
        set_threshold();
    }
    __device__ __forceinline__ void gather(bool in, float v, uint32_t token) {
        const uint64_t m = __ballot(in);
        if (!m) return;
        if (in) buf[count + __popcll(m & ((1ull << lane) - 1))] = top_key(v, token);
        count += __popcll(m);
        if (count >= 64) flush();
    }
    // first threshold: the top-th largest lane maximum
    __device__ __forceinline__ void seed(float lane_max, bool any) {
        const uint64_t s = sort64(any ? top_key(lane_max, (uint32_t)lane) : 0, lane);
        const uint64_t k = lane_value(s, top - 1);
        thr = k ? key_value(k) : -__builtin_inff();
    }
};

// What the rows' results are once the statistics and the sorted list are known.
__device__ __forceinline__ void finish_row(const LogprobArgs& a, int64_t row, const Stat& st,
                                           float target_logit, bool has_target, uint64_t list,
                                           int lane) {
    const bool empty = st.s == 0.f;  // every logit is -inf
    const float lns = empty ? 0.f : logf(st.s);
    if (lane == 0) {
        const float lse = empty ? -__builtin_inff() : fmaf(st.m, a.scale, lns);
        if (a.lse) a.lse[row] = lse;
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
    if (lane < a.top) {
        const bool some = list != 0;
        float lp = -__builtin_inff();
        if (some && !empty) lp = (key_value(list) - st.m) * a.scale - lns;
        a.top_id[row * a.top + lane] = some ? (int32_t)~(uint32_t)list : -1;
        a.top_logprob[row * a.top + lane] = lp;
    }
}

__device__ __forceinline__ Stat wave_join(Stat st, float c) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        st.join(__shfl_xor(st.m, off), __shfl_xor(st.s, off), __shfl_xor(st.T, off), c);
    return st;
}

// ---- forward ------------------------------------------------------------------------------
template <bool BF16, bool TOP>
__global__ void __launch_bounds__(64 * kLpWaves) logprob_fwd(LogprobArgs a) {
    using L = Lg<BF16>;
    using E = typename L::E;
    constexpr int N = L::N, U = 4;  // vectors a lane takes of a block
    __shared__ uint64_t s_buf[TOP ? kLpWaves : 1][TOP ? 128 : 1];
    __shared__ float s_stat[kLpWaves][3];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = (int64_t)(blockIdx.x / (uint32_t)a.splits);
    const int split = (int)(blockIdx.x % (uint32_t)a.splits);
    const E* x = static_cast<const E*>(a.logits) + row * a.ld;
    const float c = a.scale * kLog2e;
    const int64_t nvec = a.V / N;
    const int64_t v0 = nvec * split / a.splits, v1 = nvec * (split + 1) / a.splits;

    // the target's logit travels beside the row
    const int64_t target = target_of(a, row);
    float tl = 0.f;
    if (wave == 0 && target >= 0) tl = L::one(x + target);

    Stat st{kLowest, 0.f, 0.f};
    WaveTop wt;
    if constexpr (TOP) wt.init(a.top, lane, s_buf[wave]);
    bool first = true;

    // K values of the lane (those not there are -inf), tokens from `token`
    auto take = [&](auto& v, auto K, bool any, auto token) {
        constexpr int kN = decltype(K)::value;
        float mb = v[0];
#pragma unroll
        for (int e = 1; e < kN; ++e) mb = fmaxf(mb, v[e]);
        if constexpr (TOP) {
            if (first) {
                wt.seed(mb, any && mb == mb);
                first = false;
            }
            if (__any(mb >= wt.thr)) {
                const float thr = wt.thr;  // of this whole block (ties may come in any order)
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    uint32_t tok;
                    const bool in = token(e, tok) && v[e] >= thr;
                    wt.gather(in, v[e], tok);
                }
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
    auto load = [&](int64_t b, typename L::T(&r)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = b + u * 64 + lane;
            r[u] = L::load(x + (i < v1 ? i : v1 - 1) * N);
        }
    };
    int64_t b = v0 + (int64_t)wave * (64 * U);
    if (b < v1) load(b, w);
    for (; b < v1; b += 64 * U * kLpWaves) {
        const int64_t bn = b + 64 * U * kLpWaves;
        if (bn < v1) load(bn, nx);
        float v[U * N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float t[N];
            L::unpack(w[u], t);
            const bool in = b + u * 64 + lane < v1;
#pragma unroll
            for (int e = 0; e < N; ++e) v[u * N + e] = in ? t[e] : -__builtin_inff();
        }
        take(v, std::integral_constant<int, U * N>{}, b + lane < v1, [&](int e, uint32_t& tok) {
            const int64_t i = b + (e / N) * 64 + lane;
            tok = (uint32_t)(i * N + e % N);
            return i < v1;
        });
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = nx[u];
    }
    if (wave == 0 && split == a.splits - 1 && nvec * N < a.V) {  // the row's last V % N logits
        const int64_t i = nvec * N + lane;
        const bool in = i < a.V;
        float v[1] = {in ? L::one(x + i) : -__builtin_inff()};
        take(v, std::integral_constant<int, 1>{}, in, [&](int, uint32_t& tok) {
            tok = (uint32_t)i;
            return in;
        });
    }
    if constexpr (TOP) {
        if (wt.count) wt.flush();
    }
    st = wave_join(st, c);
    if (lane == 0) s_stat[wave][0] = st.m, s_stat[wave][1] = st.s, s_stat[wave][2] = st.T;
    if constexpr (TOP) s_buf[wave][lane] = wt.list;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int k = 1; k < kLpWaves; ++k) {
        st.join(s_stat[k][0], s_stat[k][1], s_stat[k][2], c);
        if constexpr (TOP) wt.list = merge64(wt.list, s_buf[k][lane], lane);
    }
    if (a.splits == 1) {
        finish_row(a, row, st, tl, target >= 0, TOP ? wt.list : 0, lane);
        return;
    }
    const int64_t at = row * a.splits + split;
    if (lane == 0) {
        a.part[at * 4] = st.m;
        a.part[at * 4 + 1] = st.s;
        a.part[at * 4 + 2] = st.T;
    }
    if constexpr (TOP) a.list[at * kMaxTop + lane] = wt.list;
}

// Joins the splits of a row (64 at most), in order.
template <bool BF16, bool TOP>
__global__ void __launch_bounds__(64 * kLpWaves) logprob_join(LogprobArgs a) {
    using L = Lg<BF16>;
    __shared__ uint64_t s_list[kLpWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x;
    const float c = a.scale * kLog2e;
    uint64_t list = 0;
    if constexpr (TOP) {
        for (int k = wave; k < a.splits; k += kLpWaves)
            list = merge64(list, a.list[(row * a.splits + k) * kMaxTop + lane], lane);
        s_list[wave][lane] = list;
        __syncthreads();
    }
    if (wave != 0) return;
    if constexpr (TOP) {
#pragma unroll
        for (int k = 1; k < kLpWaves; ++k) list = merge64(list, s_list[k][lane], lane);
    }
    const int64_t target = target_of(a, row);
    float tl = 0.f;
    if (target >= 0)
        tl = L::one(static_cast<const typename L::E*>(a.logits) + row * a.ld + target);
    Stat st{kLowest, 0.f, 0.f};
    if (lane < a.splits) {
        const float* q = a.part + (row * a.splits + lane) * 4;
        st = Stat{q[0], q[1], q[2]};
    }
    st = wave_join(st, c);
    finish_row(a, row, st, tl, target >= 0, list, lane);
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
    // about 1024 workgroups, of 4096 logits at least
    int64_t n = a.rows > 0 ? (1024 + a.rows - 1) / a.rows : 1;
    const int64_t most = (a.V + 4095) / 4096;
    if (n > most) n = most;
    if (n > 64) n = 64;
    a.splits = n < 1 ? 1 : (int)n;
    (void)bf16;
}

LogprobWs logprob_ws(const LogprobArgs& a) {
    LogprobWs w{};
    if (a.splits < 2) return w;
    const size_t n = (size_t)a.rows * (size_t)a.splits;
    w.part = 0;
    w.list = (n * 16 + 255) / 256 * 256;
    w.total = w.list + (a.top ? n * kMaxTop * 8 : 0);
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
