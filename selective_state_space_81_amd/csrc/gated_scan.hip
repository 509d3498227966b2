// gated_scan.hip -- the gated linear recurrence (ms_gated_scan_fwd / _bwd,
// ms_gated_step).  Per channel d, along the sequence:
//
//   sr = sigmoid(r), si = sigmoid(i), la = -c softplus(lam) sr, a = e^la
//   n  = sqrt(1 - a^2),  b = n si x
//   h  = A h + b,  A = a (0 where the step resets),  y = h  or  h silu(z)
//
// Gradients, with g_t = dL/dh_t = dy_t (silu z_t) + A_{t+1} g_{t+1}:
//
//   dx = g n si,  di = g n x si (1 - si),  dz = dy h silu'(z)
//   q  = la dL/dla = g (A h_{t-1} la - si x a^2 la / n)
//   dr = q (1 - sr),  dlam = sum q sigmoid(lam) / softplus(lam)
//
// q keeps la / n together: as la -> 0 the ratio goes to 0 like sqrt(-la/2),
// so the gradient stays finite where d n / d la alone does not.
//
// Layout.  A workgroup owns CH = VEC * LC neighbouring channels and kWaves
// consecutive pieces of time; lane (rg, lc) of a wave holds VEC channels at
// TAU consecutive steps, RG = 64 / LC such groups side by side in time.  Each
// lane composes its own steps into one affine map (P, H), the groups of a
// wave are joined by a shuffle scan, the waves through LDS, and the workgroup
// walks its channels along the sequence with the state in registers, so every
// input is read once and every output written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "lm_internal.h"
#include "msscan_internal.h"

namespace msscan {
namespace {

using namespace dev;

// ---- VEC io values of one row ---------------------------------------------------
// Rows of an odd channel count are aligned to their element only, so the
// vector accesses assume no more (gfx950 serves them unaligned).
template <int VEC, bool BF16>
struct RowIo;
template <>
struct RowIo<4, true> {
    typedef uint16_t E;
    typedef uint32_t T __attribute__((ext_vector_type(2)));
    typedef T M __attribute__((aligned(2)));
    static __device__ __forceinline__ void unpack(T w, float (&v)[4]) {
        v[0] = __uint_as_float(w[0] << 16);
        v[1] = __uint_as_float(w[0] & 0xffff0000u);
        v[2] = __uint_as_float(w[1] << 16);
        v[3] = __uint_as_float(w[1] & 0xffff0000u);
    }
    static __device__ __forceinline__ T pack(const float (&v)[4]) {
        auto bits = [](float f) { return (uint32_t)f32_to_bf16_rne(f); };
        return T{bits(v[0]) | (bits(v[1]) << 16), bits(v[2]) | (bits(v[3]) << 16)};
    }
};
template <>
struct RowIo<1, true> {
    typedef uint16_t E;
    typedef uint16_t T;
    typedef T M;
    static __device__ __forceinline__ void unpack(T w, float (&v)[1]) {
        v[0] = __uint_as_float((uint32_t)w << 16);
    }
    static __device__ __forceinline__ T pack(const float (&v)[1]) { return f32_to_bf16_rne(v[0]); }
};
template <>
struct RowIo<4, false> {
    typedef float E;
    typedef float T __attribute__((ext_vector_type(4)));
    typedef T M __attribute__((aligned(4)));
    static __device__ __forceinline__ void unpack(T w, float (&v)[4]) {
        v[0] = w[0], v[1] = w[1], v[2] = w[2], v[3] = w[3];
    }
    static __device__ __forceinline__ T pack(const float (&v)[4]) {
        return T{v[0], v[1], v[2], v[3]};
    }
};
template <>
struct RowIo<1, false> {
    typedef float E;
    typedef float T;
    typedef T M;
    static __device__ __forceinline__ void unpack(T w, float (&v)[1]) { v[0] = w; }
    static __device__ __forceinline__ T pack(const float (&v)[1]) { return v[0]; }
};

template <class R>
__device__ __forceinline__ typename R::T ld_row(const typename R::E* p) {
    return *reinterpret_cast<const typename R::M*>(p);
}
template <class R>
__device__ __forceinline__ void st_row(typename R::E* p, typename R::T v) {
    *reinterpret_cast<typename R::M*>(p) = v;
}

// ---- the gates of one element ------------------------------------------------------
__device__ __forceinline__ float sigmoid_f(float v) { return hw_rcp(1.f + hw_exp2(-v * kLog2e)); }

// softplus with a small relative error also where it is small (the decay rate
// of a slow channel is a softplus of 1e-3 and less).
__device__ __forceinline__ float softplus_rel(float v) {
    return v > 20.f ? v : log1pf(expf(v));
}
// sigmoid(v) / softplus(v): tends to 1 as v falls (both to e^v).
__device__ __forceinline__ float sigmoid_over_softplus(float v) {
    if (v < -16.f) return 1.f - 0.5f * expf(v);  // next term e^2v / 3: below 1e-14
    return 1.f / ((1.f + expf(-v)) * softplus_rel(v));
}

// 1 - a^2 for a = 2^la2.  With x = ln(a^2) in (-1/8, 0] the series of
// -expm1(x) to x^5 (the next term is below 3e-8 relative); further out
// 1 - a^2 itself, whose cancellation costs at most 8 rounding errors of a^2
// (5e-7 relative, halved by the root).
__device__ __forceinline__ float one_minus_square(float la2, float a) {
    const float x = la2 * (2.f * kLn2);
    float p = fmaf(x, 1.f / 120.f, 1.f / 24.f);
    p = fmaf(x, p, 1.f / 6.f);
    p = fmaf(x, p, 0.5f);
    p = fmaf(x, p, 1.f);
    return x > -0.125f ? -x * p : fmaf(-a, a, 1.f);
}

__device__ __forceinline__ float sqrt_f(float v) { return __builtin_amdgcn_sqrtf(v); }

// (P, H) applied to h.  With resets a decay of 0 cuts the past off whole: a
// NaN or infinity before the reset must not come through as 0 * NaN.
template <bool RESET>
__device__ __forceinline__ float apply(float P, float h, float H) {
    const float v = fmaf(P, h, H);
    if constexpr (RESET) return P == 0.f ? H : v;
    return v;
}

// ---- forward ------------------------------------------------------------------------
template <int VEC_, bool BF16_>
struct Shape {
    static constexpr int VEC = VEC_;
    static constexpr bool BF16 = BF16_;
    static constexpr int LC = VEC == 4 ? 8 : 32;  // lanes across channels
    static constexpr int RG = 64 / LC;            // time groups in a wave
    static constexpr int CH = VEC * LC;           // channels of a workgroup
};
constexpr int kWaves = 4;

// Lane geometry shared by the passes.
template <class S>
struct Lane {
    int lane, wave, rg, lc, b, ch;
    bool live;     // the lane's channels exist
    int64_t base;  // element offset of (b, 0, ch)
    __device__ __forceinline__ Lane(const GatedArgs& a) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        rg = lane / S::LC;
        lc = lane % S::LC;
        const uint32_t tiles = ((uint32_t)a.Dn + S::CH - 1) / S::CH;
        const uint32_t l = xcd_logical(blockIdx.x, gridDim.x);
        b = (int)(l / tiles);
        ch = (int)(l % tiles) * S::CH + lc * S::VEC;
        live = ch < a.Dn;
        // The last lane of a channel count that VEC does not divide takes the
        // last VEC channels; some are its neighbour's too, and both store the
        // same values.  Lanes past it read them and store nothing.
        ch = min(ch, a.Dn - S::VEC);
        base = (int64_t)b * a.L * a.Dn + ch;
    }
};

template <int VEC, bool BF16, bool GATE, bool RESET>
__global__ void __launch_bounds__(64 * kWaves) gated_fwd(GatedArgs a) {
    using S = Shape<VEC, BF16>;
    using R = RowIo<VEC, BF16>;
    using T = typename R::T;
    constexpr int TAU = VEC == 4 ? 8 : 16;
    constexpr int LC = S::LC, RG = S::RG, TW = TAU * RG, TB = TW * kWaves;
    static_assert(TW % kGatedBlock == 0, "a wave starts at a saved state");
    __shared__ float2 s_sum[2][kWaves][S::CH];
    const Lane<S> g(a);
    using E = typename R::E;
    const E* px = static_cast<const E*>(a.x) + g.base;
    const E* pr = static_cast<const E*>(a.r) + g.base;
    const E* pi = static_cast<const E*>(a.i) + g.base;
    const E* pz = static_cast<const E*>(a.z) + g.base;
    E* py = static_cast<E*>(a.y) + g.base;
    const int64_t rs = a.Dn;

    float k[VEC], carry[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        k[c] = -a.sharp * kLog2e * softplus_rel(a.lam[g.ch + c]);
        carry[c] = a.h0 ? a.h0[(int64_t)g.b * a.Dn + g.ch + c] : 0.f;
    }

    T rx[TAU], rr[TAU], ri[TAU], rz[TAU];
    auto load = [&](int64_t t0, const E* p, T(&w)[TAU]) {
#pragma unroll
        for (int j = 0; j < TAU; ++j) w[j] = ld_row<R>(p + min(t0 + j, a.L - 1) * rs);
    };
    int64_t t0 = (int64_t)g.wave * TW + g.rg * TAU;  // the lane's first step
    load(t0, px, rx);
    load(t0, pr, rr);
    load(t0, pi, ri);
    if constexpr (GATE) load(t0, pz, rz);

    int par = 0;
    for (int64_t tb = 0; tb < a.L; tb += TB, t0 += TB, par ^= 1) {
        // the lane's steps as A[j], B[j] and composed as (P, H)
        float A[TAU][VEC], B[TAU][VEC], P[VEC], H[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) P[c] = 1.f, H[c] = 0.f;
#pragma unroll
        for (int j = 0; j < TAU; ++j) {
            const bool in = t0 + j < a.L;
            bool cut = false;
            if constexpr (RESET) cut = in && a.reset[(int64_t)g.b * a.L + t0 + j] != 0;
            float x[VEC], r[VEC], i[VEC];
            R::unpack(rx[j], x);
            R::unpack(rr[j], r);
            R::unpack(ri[j], i);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float la2 = k[c] * sigmoid_f(r[c]);
                const float e = hw_exp2(la2);
                const float n = sqrt_f(one_minus_square(la2, e));
                A[j][c] = in ? (cut ? 0.f : e) : 1.f;
                B[j][c] = in ? n * sigmoid_f(i[c]) * x[c] : 0.f;
                H[c] = apply<RESET>(A[j][c], H[c], B[j][c]);
                P[c] *= A[j][c];
            }
        }
        if (tb + TB < a.L) {  // the next block's inputs travel during the exchange below
            load(t0 + TB, px, rx);
            load(t0 + TB, pr, rr);
            load(t0 + TB, pi, ri);
        }
        // inclusive scan over the wave's time groups, then the wave's total to LDS
#pragma unroll
        for (int off = LC; off < 64; off <<= 1) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float Pu = __shfl_up(P[c], off), Hu = __shfl_up(H[c], off);
                if (g.lane >= off) {
                    H[c] = apply<RESET>(P[c], Hu, H[c]);
                    P[c] *= Pu;
                }
            }
        }
        if (g.rg == RG - 1) {
#pragma unroll
            for (int c = 0; c < VEC; ++c)
                s_sum[par][g.wave][g.lc * VEC + c] = make_float2(P[c], H[c]);
        }
        float h[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {  // exclusive
            P[c] = __shfl_up(P[c], LC);
            H[c] = __shfl_up(H[c], LC);
            if (g.rg == 0) P[c] = 1.f, H[c] = 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w == g.wave) {
#pragma unroll
                for (int c = 0; c < VEC; ++c) h[c] = apply<RESET>(P[c], carry[c], H[c]);
            }
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float2 q = s_sum[par][w][g.lc * VEC + c];
                carry[c] = apply<RESET>(q.x, carry[c], q.y);
            }
        }
        if (a.states && g.live && t0 % kGatedBlock == 0 && t0 < a.L) {
            float* st = a.states + ((int64_t)g.b * a.nstates + t0 / kGatedBlock) * a.Dn + g.ch;
#pragma unroll
            for (int c = 0; c < VEC; ++c) st[c] = h[c];
        }
#pragma unroll
        for (int j = 0; j < TAU; ++j) {
            float o[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                h[c] = apply<RESET>(A[j][c], h[c], B[j][c]);
                o[c] = h[c];
            }
            if constexpr (GATE) {
                float z[VEC];
                R::unpack(rz[j], z);
#pragma unroll
                for (int c = 0; c < VEC; ++c) o[c] *= silu_f(z[c]);
            }
            if (g.live && t0 + j < a.L) st_row<R>(py + (t0 + j) * rs, R::pack(o));
        }
        if constexpr (GATE) {
            if (tb + TB < a.L) load(t0 + TB, pz, rz);
        }
    }
    if (a.h_last && g.live && g.wave == 0 && g.rg == 0) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) a.h_last[(int64_t)g.b * a.Dn + g.ch + c] = carry[c];
    }
}

// ---- backward -----------------------------------------------------------------------
// The same walk from the end of the sequence.  Each wave starts its forward
// recurrence from the state saved before its first step, so only the message
// A_t g_t travels between waves (through LDS) and blocks (in registers).
template <int VEC, bool BF16, bool GATE, bool RESET>
__global__ void __launch_bounds__(64 * kWaves) gated_bwd(GatedArgs a) {
    using S = Shape<VEC, BF16>;
    using R = RowIo<VEC, BF16>;
    using T = typename R::T;
    using E = typename R::E;
    constexpr int TAU = VEC == 4 ? 4 : 16;
    constexpr int LC = S::LC, RG = S::RG, TW = TAU * RG, TB = TW * kWaves;
    static_assert(TW == kGatedBlock, "a wave starts at a saved state");
    __shared__ float2 s_sum[2][kWaves][S::CH];
    __shared__ float s_lam[kWaves][S::CH];
    const Lane<S> g(a);
    auto in_ptr = [&](const void* p) { return static_cast<const E*>(p) + g.base; };
    auto out_ptr = [&](void* p) { return static_cast<E*>(p) + g.base; };
    const E *px = in_ptr(a.x), *pr = in_ptr(a.r), *pi = in_ptr(a.i), *pz = in_ptr(a.z),
            *pg = in_ptr(a.dy);
    E *ox = out_ptr(a.dx), *orr = out_ptr(a.dr), *oi = out_ptr(a.di), *oz = out_ptr(a.dz);
    const int64_t rs = a.Dn;

    float k[VEC], carry[VEC], dlam[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        k[c] = -a.sharp * kLog2e * softplus_rel(a.lam[g.ch + c]);
        carry[c] = a.dh_last ? a.dh_last[(int64_t)g.b * a.Dn + g.ch + c] : 0.f;
        dlam[c] = 0.f;
    }
    int par = 0;
    const int64_t nb = (a.L + TB - 1) / TB;
    for (int64_t blk = nb - 1; blk >= 0; --blk, par ^= 1) {
        const int64_t tw = blk * TB + g.wave * TW;  // the wave's first step
        const int64_t t0 = tw + g.rg * TAU;
        T rx[TAU], rr[TAU], ri[TAU], rz[TAU], rg_[TAU];
#pragma unroll
        for (int j = 0; j < TAU; ++j) {
            const int64_t o = min(t0 + j, a.L - 1) * rs;
            rx[j] = ld_row<R>(px + o);
            rr[j] = ld_row<R>(pr + o);
            ri[j] = ld_row<R>(pi + o);
            rg_[j] = ld_row<R>(pg + o);
            if constexpr (GATE) rz[j] = ld_row<R>(pz + o);
        }
        // forward: A, h_{t-1}
        float sr[TAU][VEC], e[TAU][VEC], A[TAU][VEC], hp[TAU][VEC], n[TAU][VEC], si[TAU][VEC];
        float P[VEC], H[VEC], h[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) P[c] = 1.f, H[c] = 0.f;
        bool in[TAU];
#pragma unroll
        for (int j = 0; j < TAU; ++j) {
            in[j] = t0 + j < a.L;
            bool cut = false;
            if constexpr (RESET) cut = in[j] && a.reset[(int64_t)g.b * a.L + t0 + j] != 0;
            float x[VEC], r[VEC], i[VEC];
            R::unpack(rx[j], x);
            R::unpack(rr[j], r);
            R::unpack(ri[j], i);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                sr[j][c] = sigmoid_f(r[c]);
                si[j][c] = sigmoid_f(i[c]);
                const float la2 = k[c] * sr[j][c];
                e[j][c] = hw_exp2(la2);
                n[j][c] = sqrt_f(one_minus_square(la2, e[j][c]));
                A[j][c] = in[j] ? (cut ? 0.f : e[j][c]) : 1.f;
                H[c] = apply<RESET>(A[j][c], H[c], in[j] ? n[j][c] * si[j][c] * x[c] : 0.f);
                P[c] *= A[j][c];
            }
        }
#pragma unroll
        for (int off = LC; off < 64; off <<= 1) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float Pu = __shfl_up(P[c], off), Hu = __shfl_up(H[c], off);
                if (g.lane >= off) {
                    H[c] = apply<RESET>(P[c], Hu, H[c]);
                    P[c] *= Pu;
                }
            }
        }
        {
            const int64_t sb = min(tw / kGatedBlock, a.nstates - 1);  // past the end: unused
            const float* st = a.states + ((int64_t)g.b * a.nstates + sb) * a.Dn + g.ch;
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                float Pe = __shfl_up(P[c], LC), He = __shfl_up(H[c], LC);
                if (g.rg == 0) Pe = 1.f, He = 0.f;
                h[c] = apply<RESET>(Pe, st[c], He);
            }
        }
        // h_{t-1} of every step, dz, and the gradient arriving at h_t from y_t
        float gh[TAU][VEC];
#pragma unroll
        for (int j = 0; j < TAU; ++j) {
            float x[VEC], dy[VEC];
            R::unpack(rx[j], x);
            R::unpack(rg_[j], dy);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                hp[j][c] = h[c];
                h[c] = apply<RESET>(A[j][c], h[c], in[j] ? n[j][c] * si[j][c] * x[c] : 0.f);
                gh[j][c] = in[j] ? dy[c] : 0.f;
            }
            if constexpr (GATE) {
                float z[VEC], dz[VEC];
                R::unpack(rz[j], z);
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    const float sz = sigmoid_f(z[c]);
                    dz[c] = dy[c] * h[c] * sz * fmaf(z[c], 1.f - sz, 1.f);
                    gh[j][c] *= z[c] * sz;
                    if (!in[j]) gh[j][c] = 0.f;
                }
                if (g.live && in[j]) st_row<R>(oz + (t0 + j) * rs, R::pack(dz));
            }
        }
        // the message to the step before the lane: c_out = P c_in + C
        float C[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) P[c] = 1.f, C[c] = 0.f;
#pragma unroll
        for (int j = TAU - 1; j >= 0; --j) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                C[c] = apply<RESET>(A[j][c], gh[j][c] + C[c], 0.f);
                P[c] *= A[j][c];
            }
        }
#pragma unroll
        for (int off = LC; off < 64; off <<= 1) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float Pd = __shfl_down(P[c], off), Cd = __shfl_down(C[c], off);
                if (g.lane + off < 64) {
                    C[c] = apply<RESET>(P[c], Cd, C[c]);
                    P[c] *= Pd;
                }
            }
        }
        if (g.rg == 0) {
#pragma unroll
            for (int c = 0; c < VEC; ++c)
                s_sum[par][g.wave][g.lc * VEC + c] = make_float2(P[c], C[c]);
        }
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            P[c] = __shfl_down(P[c], LC);
            C[c] = __shfl_down(C[c], LC);
            if (g.rg == RG - 1) P[c] = 1.f, C[c] = 0.f;
        }
        __syncthreads();
        float m[VEC];  // the message arriving from the step after the lane's last
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
            if (w == g.wave) {
#pragma unroll
                for (int c = 0; c < VEC; ++c) m[c] = apply<RESET>(P[c], carry[c], C[c]);
            }
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float2 q = s_sum[par][w][g.lc * VEC + c];
                carry[c] = apply<RESET>(q.x, carry[c], q.y);
            }
        }
#pragma unroll
        for (int j = TAU - 1; j >= 0; --j) {
            float x[VEC], dx[VEC], dr[VEC], di[VEC];
            R::unpack(rx[j], x);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float gt = gh[j][c] + m[c];  // dL/dh_t
                m[c] = apply<RESET>(A[j][c], gt, 0.f);
                const float s = si[j][c], la = k[c] * kLn2 * sr[j][c];
                const float ratio = n[j][c] > 0.f ? la * hw_rcp(n[j][c]) : 0.f;
                const float keep = apply<RESET>(A[j][c], hp[j][c], 0.f) * la;
                const float q = gt * fmaf(-s * x[c] * e[j][c], e[j][c] * ratio, keep);
                dx[c] = gt * n[j][c] * s;
                di[c] = dx[c] * x[c] * (1.f - s);
                dr[c] = q * (1.f - sr[j][c]);
                dlam[c] += in[j] ? q : 0.f;
            }
            if (g.live && in[j]) {
                st_row<R>(ox + (t0 + j) * rs, R::pack(dx));
                st_row<R>(orr + (t0 + j) * rs, R::pack(dr));
                st_row<R>(oi + (t0 + j) * rs, R::pack(di));
            }
        }
    }
    if (a.dh0 && g.live && g.wave == 0 && g.rg == 0) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) a.dh0[(int64_t)g.b * a.Dn + g.ch + c] = carry[c];
    }
    // sum of q over the lane groups (shuffles) and the waves (LDS)
#pragma unroll
    for (int off = LC; off < 64; off <<= 1)
#pragma unroll
        for (int c = 0; c < VEC; ++c) dlam[c] += __shfl_xor(dlam[c], off);
    if (g.rg == 0) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) s_lam[g.wave][g.lc * VEC + c] = dlam[c];
    }
    __syncthreads();
    if (g.live && g.wave == 0 && g.rg == 0) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += s_lam[w][g.lc * VEC + c];
            a.part[(int64_t)g.b * a.Dn + g.ch + c] = v;
        }
    }
}

// dlam[d] = sigmoid/softplus(lam) * sum of the partials, in order
__global__ void __launch_bounds__(256) gated_dlam(GatedArgs a, int64_t rows) {
    const int d = blockIdx.x * 256 + threadIdx.x;
    if (d >= a.Dn) return;
    float v = 0.f;
    for (int64_t i = 0; i < rows; ++i) v += a.part[i * a.Dn + d];
    a.dlam[d] = v * sigmoid_over_softplus(a.lam[d]);
}

// ---- one step ------------------------------------------------------------------------
template <int VEC, bool BF16>
__global__ void __launch_bounds__(256) gated_step(GatedArgs a, int64_t nvec) {
    using R = RowIo<VEC, BF16>;
    using T = typename R::T;
    typedef float F __attribute__((ext_vector_type(VEC)));
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= nvec) return;
    const int d = (int)(v % (uint32_t)(a.Dn / VEC)) * VEC;
    float x[VEC], r[VEC], i[VEC], o[VEC];
    float* hp = a.h_last + v * VEC;
    F h = *reinterpret_cast<const F*>(hp);
    R::unpack(static_cast<const T*>(a.x)[v], x);
    R::unpack(static_cast<const T*>(a.r)[v], r);
    R::unpack(static_cast<const T*>(a.i)[v], i);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        const float la2 = -a.sharp * kLog2e * softplus_rel(a.lam[d + c]) * sigmoid_f(r[c]);
        const float e = hw_exp2(la2);
        const float n = sqrt_f(one_minus_square(la2, e));
        o[c] = fmaf(e, h[c], n * sigmoid_f(i[c]) * x[c]);
        h[c] = o[c];
    }
    *reinterpret_cast<F*>(hp) = h;
    if (a.z) {
        float z[VEC];
        R::unpack(static_cast<const T*>(a.z)[v], z);
#pragma unroll
        for (int c = 0; c < VEC; ++c) o[c] *= silu_f(z[c]);
    }
    static_cast<T*>(a.y)[v] = R::pack(o);
}

template <int VEC, bool BF16>
unsigned gated_grid(const GatedArgs& a) {
    constexpr int CH = Shape<VEC, BF16>::CH;
    return (unsigned)((a.Dn + CH - 1) / CH) * (unsigned)a.batch;
}

template <int VEC, bool BF16>
void fwd_variant(const GatedArgs& a, hipStream_t s) {
    const dim3 grid(gated_grid<VEC, BF16>(a)), blk(64 * kWaves);
    if (a.z && a.reset) hipLaunchKernelGGL((gated_fwd<VEC, BF16, true, true>), grid, blk, 0, s, a);
    else if (a.z) hipLaunchKernelGGL((gated_fwd<VEC, BF16, true, false>), grid, blk, 0, s, a);
    else if (a.reset) hipLaunchKernelGGL((gated_fwd<VEC, BF16, false, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((gated_fwd<VEC, BF16, false, false>), grid, blk, 0, s, a);
}

template <int VEC, bool BF16>
void bwd_variant(const GatedArgs& a, hipStream_t s) {
    const dim3 grid(gated_grid<VEC, BF16>(a)), blk(64 * kWaves);
    if (a.z && a.reset) hipLaunchKernelGGL((gated_bwd<VEC, BF16, true, true>), grid, blk, 0, s, a);
    else if (a.z) hipLaunchKernelGGL((gated_bwd<VEC, BF16, true, false>), grid, blk, 0, s, a);
    else if (a.reset) hipLaunchKernelGGL((gated_bwd<VEC, BF16, false, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((gated_bwd<VEC, BF16, false, false>), grid, blk, 0, s, a);
}

}  // namespace

// Four channels a lane wherever there are four.  (h_last over h0 with a
// channel count that four does not divide: a workgroup may store a shared
// channel's h_last before its neighbour has read the h0 there.)
static bool four_channels(const GatedArgs& a) {
    return a.Dn % 4 == 0 || (a.Dn >= 4 && (!a.h0 || a.h0 != a.h_last));
}

size_t gated_bwd_part_floats(int batch, int64_t, int Dn) { return (size_t)batch * (size_t)Dn; }

hipError_t launch_gated_fwd(const GatedArgs& a, bool bf16, hipStream_t s) {
    ProfScope ps(s, kPhaseMain);
    if (four_channels(a)) bf16 ? fwd_variant<4, true>(a, s) : fwd_variant<4, false>(a, s);
    else bf16 ? fwd_variant<1, true>(a, s) : fwd_variant<1, false>(a, s);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedArgs& a, bool bf16, hipStream_t s) {
    {
        ProfScope ps(s, kPhaseMain);
        if (four_channels(a)) bf16 ? bwd_variant<4, true>(a, s) : bwd_variant<4, false>(a, s);
        else bf16 ? bwd_variant<1, true>(a, s) : bwd_variant<1, false>(a, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ProfScope ps(s, kPhaseReduce);
    hipLaunchKernelGGL(gated_dlam, dim3((a.Dn + 255) / 256), dim3(256), 0, s, a, (int64_t)a.batch);
    return hipGetLastError();
}

hipError_t launch_gated_step(const GatedArgs& a, bool bf16, hipStream_t s) {
    ProfScope ps(s, kPhaseStep);
    const int vec = a.Dn % 4 == 0 ? 4 : 1;
    const int64_t nvec = (int64_t)a.batch * (a.Dn / vec);
    const dim3 grid((unsigned)((nvec + 255) / 256)), blk(256);
    if (vec == 4) {
        if (bf16) hipLaunchKernelGGL((gated_step<4, true>), grid, blk, 0, s, a, nvec);
        else hipLaunchKernelGGL((gated_step<4, false>), grid, blk, 0, s, a, nvec);
    } else {
        if (bf16) hipLaunchKernelGGL((gated_step<1, true>), grid, blk, 0, s, a, nvec);
        else hipLaunchKernelGGL((gated_step<1, false>), grid, blk, 0, s, a, nvec);
    }
    return hipGetLastError();
}

}  // namespace msscan
