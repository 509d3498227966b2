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
// Layout.  A workgroup owns CH = VEC * LC neighbouring channels and one block
// of time, a wave a piece of it; lane (rg, lc) holds VEC channels at TAU
// consecutive steps, RG = 64 / LC such groups side by side in time.  Each lane
// composes its own steps into one affine map (P, H), the groups of a wave are
// joined by a shuffle scan, the waves through LDS and the blocks by look-back
// (Chain below), so every input is read once and every output written once
// whatever the number of channels.
//
// What bounds it: bytes, with the arithmetic close behind (42 instructions an
// element forward, 8 of them transcendental; 90 backward).  At 8 x 2048 x 1536
// bf16 with the gate the forward moves 252 MB in 58 us (4.3 TB/s of the 5.6
// that a copy reaches) and keeps the vector units busy for half of that.  The
// backward moves 466 MB in 100 us.  One sequence of 131072 x 1536, no gate: 1.61
// GB in 333 us, of which 25 are waiting for the block before.
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
struct RowIo;  // out(): every value -infinity
template <>
struct RowIo<4, true> {
    typedef uint16_t E;
    typedef uint32_t T __attribute__((ext_vector_type(2)));
    typedef T M __attribute__((aligned(2)));
    static __device__ __forceinline__ T out() { return T{0xff80ff80u, 0xff80ff80u}; }
    static __device__ __forceinline__ void unpack(T w, float (&v)[4]) {
        v[0] = __uint_as_float(w[0] << 16);
        v[1] = __uint_as_float(w[0] & 0xffff0000u);
        v[2] = __uint_as_float(w[1] << 16);
        v[3] = __uint_as_float(w[1] & 0xffff0000u);
    }
    static __device__ __forceinline__ T pack(const float (&v)[4]) {
        typedef float F __attribute__((ext_vector_type(4)));
        typedef __bf16 B __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(T, __builtin_convertvector((F{v[0], v[1], v[2], v[3]}), B));
    }
};
template <>
struct RowIo<2, true> {
    typedef uint16_t E;
    typedef uint32_t T;
    typedef T M __attribute__((aligned(2)));
    static __device__ __forceinline__ T out() { return 0xff80ff80u; }
    static __device__ __forceinline__ void unpack(T w, float (&v)[2]) {
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ T pack(const float (&v)[2]) {
        typedef float F __attribute__((ext_vector_type(2)));
        typedef __bf16 B __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(T, __builtin_convertvector((F{v[0], v[1]}), B));
    }
};
template <>
struct RowIo<2, false> {
    typedef float E;
    typedef float T __attribute__((ext_vector_type(2)));
    typedef T M __attribute__((aligned(4)));
    static __device__ __forceinline__ T out() {
        const float f = -__builtin_inff();
        return T{f, f};
    }
    static __device__ __forceinline__ void unpack(T w, float (&v)[2]) { v[0] = w[0], v[1] = w[1]; }
    static __device__ __forceinline__ T pack(const float (&v)[2]) { return T{v[0], v[1]}; }
};
template <>
struct RowIo<1, true> {
    typedef uint16_t E;
    typedef uint16_t T;
    typedef T M;
    static __device__ __forceinline__ T out() { return 0xff80; }
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
    static __device__ __forceinline__ T out() {
        const float f = -__builtin_inff();
        return T{f, f, f, f};
    }
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
    static __device__ __forceinline__ T out() { return -__builtin_inff(); }
    static __device__ __forceinline__ void unpack(T w, float (&v)[1]) { v[0] = w; }
    static __device__ __forceinline__ T pack(const float (&v)[1]) { return v[0]; }
};

template <class R>
__device__ __forceinline__ typename R::T ld_row(const char* row, uint32_t off) {
    return *reinterpret_cast<const typename R::M*>(row + off);
}
// Written once and not read here: non-temporal (131072 x 1536 366 -> 361 us, a
// training pass of 8 x 2048 x 1536 200 -> 194; such loads gained nothing).
template <class R>
__device__ __forceinline__ void st_row(char* row, uint32_t off, typename R::T v) {
    __builtin_nontemporal_store(v, reinterpret_cast<typename R::M*>(row + off));
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

// 1 - a^2 for a = 2^t.  For ln(a^2) in (-1/8, 0] -t times a cubic in t fitted
// to (1 - 4^t) / -t there (Chebyshev nodes, 1.6e-08 relative); further out
// 1 - a^2 itself, whose cancellation costs at most 8 rounding errors of a^2
// (5e-7 relative, halved by the root).
constexpr float kSquareNear = 0.0901684401f;
__device__ __forceinline__ float one_minus_square(float t, float a) {
    float p = fmaf(t, 0.146416157f, 0.443615764f);
    p = fmaf(t, p, 0.960898519f);
    p = fmaf(t, p, 1.38629436f);
    return t > -kSquareNear ? -t * p : fmaf(-a, a, 1.f);
}

__device__ __forceinline__ float sqrt_f(float v) { return __builtin_amdgcn_sqrtf(v); }

// With resets a step that resets, or whose own decay is exactly 0, has the decay
// kCut: a product of decays that falls to 0 must not pass for one, and a 0 would
// let a NaN or infinity before the reset through as 0 * NaN.
constexpr float kCut = -1.f;

// (P, H) applied to h.
template <bool RESET>
__device__ __forceinline__ float apply(float P, float h, float H) {
    const float v = fmaf(P, h, H);
    if constexpr (RESET) return P < 0.f ? H : v;
    return v;
}

// The decay of two maps in a row: the product, which is at most each of them,
// or kCut where one cuts (then that is the least of the three).  A NaN may be
// lost to the other's number here: the H of its map is NaN as well.
template <bool RESET>
__device__ __forceinline__ float both(float P, float Q) {
    const float v = P * Q;
    if constexpr (RESET) return fminf(fminf(P, Q), v);
    return v;
}

// The decay of a step.
template <bool RESET>
__device__ __forceinline__ float decay(float e, bool cut) {
    if constexpr (RESET) return cut || e == 0.f ? kCut : e;
    return e;
}

// ---- geometry -----------------------------------------------------------------------
// VEC channels and TAU steps a lane, LC lanes across channels, W waves along
// time.  A workgroup takes one block of TB steps and gets the state before it
// from the workgroups of earlier blocks (see Chain).
template <int VEC_, int LC_, int TAU_, int W_, bool BF16_>
struct Geo {
    static constexpr int VEC = VEC_, LC = LC_, TAU = TAU_, W = W_;
    static constexpr bool BF16 = BF16_;
    static constexpr int RG = 64 / LC;         // time groups in a wave
    static constexpr int CH = VEC * LC;        // channels of a workgroup
    static constexpr int TW = TAU * RG;        // steps of a wave
    static constexpr int TB = TW * W;          // steps of a workgroup
    static_assert(TW % kGatedBlock == 0, "a wave starts at a saved state");
};

// Channel tiles of a batch row; a chain is one tile of one batch row.
template <class G>
__device__ __forceinline__ uint32_t tiles_of(const GatedArgs& a) {
    return ((uint32_t)a.Dn + G::CH - 1) / G::CH;
}

// Lane geometry of chain `chain`.
template <class G>
struct Lane {
    int lane, wave, rg, lc, b, ch;
    bool live;    // the lane's channels exist
    uint32_t chb;        // byte offset of the lane's channels
    uint32_t rowb, inb;  // bytes from one row to the next: of x, r, i and z inb
    __device__ __forceinline__ Lane(const GatedArgs& a, uint32_t chain) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        rg = lane / G::LC;
        lc = lane % G::LC;
        const uint32_t tiles = tiles_of<G>(a);
        b = (int)(chain / tiles);
        ch = (int)(chain % tiles) * G::CH + lc * G::VEC;
        live = ch < a.Dn;
        // The last lane of a channel count that VEC does not divide takes the
        // last VEC channels; some are its neighbour's too, and both store the
        // same values.  Lanes past it read them and store nothing.
        ch = min(ch, a.Dn - G::VEC);
        constexpr int E = G::BF16 ? 2 : 4;
        chb = (uint32_t)ch * E;
        rowb = (uint32_t)a.Dn * E;  // both below 2^24 (the entry points check)
        inb = (uint32_t)a.ld * E;
    }
    // Byte offset of the lane's step j within its wave's TW steps, of which
    // `left` exist (reads past them repeat the last one), in rows `pitch` apart.
    __device__ __forceinline__ uint32_t at(int j, int left, uint32_t pitch) const {
        return __umul24((uint32_t)min(rg * G::TAU + j, left - 1), pitch) + chb;
    }
    // Address of step t of the wave's batch row (wave-uniform).
    template <class P>
    __device__ __forceinline__ auto row(const GatedArgs& a, P* p, int64_t t, uint32_t pitch) const {
        typedef typename std::conditional<std::is_const<P>::value, const char, char>::type C;
        return static_cast<C*>(p) + ((int64_t)b * a.L + t) * pitch;
    }
};

// Where a wave's steps are in block blk (the same for every chain).
template <class G>
struct Place {
    int64_t tw, tr;  // its first step; that step, or the last of all where it is past the end
    int left;        // steps from tr on that exist, TW at most
    bool ragged;     // not all of the wave's steps exist
    int own;         // how many do (<= 0: none)
    __device__ __forceinline__ Place(const GatedArgs& a, int64_t blk) {
        tw = blk * G::TB + (int64_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * G::TW;
        tr = min(tw, a.L - 1);
        left = (int)min(a.L - tr, (int64_t)G::TW);
        own = (int)min(a.L - tw, (int64_t)G::TW);
        ragged = own < G::TW;
    }
    __device__ __forceinline__ int mine(const Lane<G>& g) const { return own - g.rg * G::TAU; }
};

// The channel of a chain's slot (lane lc's channel c is slot lc * VEC + c).
template <class G>
__device__ __forceinline__ int slot_channel(const GatedArgs& a, uint32_t chain, int slot) {
    const int ch = (int)(chain % tiles_of<G>(a)) * G::CH + slot / G::VEC * G::VEC;
    return min(ch, a.Dn - G::VEC) + slot % G::VEC;
}

// ---- the state between blocks -----------------------------------------------------------
// Blocks of one chain run on different workgroups.  Each publishes what it
// does to a state, (P, H), as soon as it has read its inputs, and the state
// after it once it knows the one before; a block looks back over up to
// kWindow others for the nearest published state and applies the (P, H)
// between in order, so the result is that of a serial chain whatever the
// timing.  As many workgroups as a chain has blocks come for its blocks, and a
// counter hands them out, earlier blocks first: a block that is waited for has
// been started, and waits for earlier ones only, so every wait ends.  (A
// counter for each chain: one for all hands out a block each 12 ns, and the
// kernel waited for it.  Chains move over the XCDs from block to block: where
// each stayed on one, their times drifted apart and rows were read in pieces.
// 8 x 2048 x 1536: 66 -> 60 us, its backward 118 -> 111, 131072 x 1536: 363 ->
// 345.)  A word of all ones is not yet published (the preparing kernel writes
// it; published NaNs have other patterns, also than kState).  The words are
// single relaxed atomics at device scope: each carries its whole message, so
// no fence orders anything else.
constexpr uint32_t kNotYet = 0xffffffffu, kState = 0xfffffffeu;
// One sequence of 131072 steps at 64 channels is bound by this chain of
// messages: 173 us with a window of 4, 117 with 8; 16 spill in the backward.
constexpr int kWindow = 8;
constexpr int kTicketStride = 16;  // words: a counter has 64 bytes to itself

__device__ __forceinline__ float plain_nan(float v) { return v == v ? v : __builtin_nanf(""); }

// Messages of one chain, one a channel: [block][CH], in the order blocks are taken.
template <int CH>
struct Chain {
    uint64_t* word;  // this lane's channel of the chain's first block

    __device__ __forceinline__ void publish(int64_t blk, uint32_t low, float high) const {
        const uint64_t w = ((uint64_t)__float_as_uint(plain_nan(high)) << 32) | low;
        __hip_atomic_store(word + blk * CH, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ void publish_map(int64_t blk, float P, float H) const {
        publish(blk, __float_as_uint(plain_nan(P)), H);
    }
    __device__ __forceinline__ void publish_state(int64_t blk, float h) const {
        publish(blk, kState, h);
    }
    // The state before block blk >= 1.  The first block publishes a state and
    // never a map, so what the window holds before it (another chain's words,
    // or the room left in front of the first) is never taken.
    template <bool RESET>
    __device__ __forceinline__ float before(int64_t blk) const {
        const uint64_t* p = word + (blk - 1) * CH;
        for (;;) {
            uint64_t w[kWindow];
#pragma unroll
            for (int k = 0; k < kWindow; ++k)
                w[k] = __hip_atomic_load(p - k * CH, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // nearest state; every message nearer than it has to be there
            int at = -1;
            bool whole = true;
#pragma unroll
            for (int k = 0; k < kWindow; ++k) {
                if (at < 0 && whole && (uint32_t)w[k] == kState) at = k;
                whole = whole && (uint32_t)w[k] != kNotYet;
            }
            if (at >= 0) {
                float h = 0.f;
#pragma unroll
                for (int k = kWindow - 1; k >= 0; --k) {
                    const float high = __uint_as_float((uint32_t)(w[k] >> 32));
                    if (k == at) h = high;
                    if (k < at) h = apply<RESET>(__uint_as_float((uint32_t)w[k]), h, high);
                }
                return h;
            }
            __builtin_amdgcn_s_sleep(1);
        }
    }
};

template <class G>
__device__ __forceinline__ Chain<G::CH> chain_of(const GatedArgs& a, uint32_t chain) {
    return Chain<G::CH>{a.word + (int64_t)chain * a.blocks * G::CH + threadIdx.x};
}

// Nothing published, no work handed out.
__global__ void __launch_bounds__(256) gated_prepare(GatedArgs a, int64_t words) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)gridDim.x * 256;
    for (int64_t k = t; k < words; k += n) a.word[k] = ~(uint64_t)0;
    for (int64_t k = t; k < a.chains; k += n) a.ticket[k * kTicketStride] = 0;
}

__global__ void __launch_bounds__(256) gated_copy(const float* from, float* to, int64_t n) {
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256)
        to[k] = from[k];
}

// This workgroup's chain, and its turn in it.
struct Work {
    uint32_t chain;
    int64_t turn;
};
__device__ __forceinline__ Work take_work(const GatedArgs& a) {
    if (a.blocks == 1) return Work{blockIdx.x, 0};
    __shared__ uint32_t s_ticket;
    const uint32_t round = blockIdx.x / a.chains, chain = (blockIdx.x + round) % a.chains;
    if (threadIdx.x == 0) s_ticket = atomicAdd(a.ticket + (size_t)chain * kTicketStride, 1u);
    __syncthreads();
    return Work{chain, __builtin_amdgcn_readfirstlane(s_ticket)};
}

// -c log2 e softplus(lam) of the workgroup's channels, one a thread, for all
// lanes through LDS (the logarithm would cost each lane VEC times over).
template <class G>
__device__ __forceinline__ void share_rates(const GatedArgs& a, uint32_t chain,
                                            float (&s_k)[G::CH]) {
    if (threadIdx.x < G::CH)
        s_k[threadIdx.x] = -a.sharp * kLog2e *
                           softplus_rel(a.lam[slot_channel<G>(a, chain, (int)threadIdx.x)]);
}

// Steps past the end of the sequence are given gates and inputs that make
// them the identity: r = -infinity is a decay of exactly 1, and x = 0.
template <class R, int TAU>
__device__ __forceinline__ void pad_steps(int mine, typename R::T (&r)[TAU],
                                          typename R::T (&x)[TAU]) {
#pragma unroll
    for (int j = 0; j < TAU; ++j)
        if (j >= mine) r[j] = R::out(), x[j] = typename R::T{};
}

// ---- forward ------------------------------------------------------------------------
template <class G, bool GATE, bool RESET>
__global__ void __launch_bounds__(64 * G::W, G::BF16 ? 3 : 2) gated_fwd(GatedArgs a) {
    constexpr int VEC = G::VEC, LC = G::LC, RG = G::RG, TAU = G::TAU, TW = G::TW, TB = G::TB,
                  W = G::W;
    using R = RowIo<VEC, G::BF16>;
    using T = typename R::T;
    __shared__ float2 s_sum[W][G::CH];
    __shared__ float s_h[G::CH], s_k[G::CH];
    const Work wk = take_work(a);
    const uint32_t chain = wk.chain;
    const int64_t blk = wk.turn;
    const bool last = blk == a.blocks - 1;
    const Lane<G> g(a, chain);
    const Place<G> pl(a, blk);
    const int mine = pl.mine(g);

    T rx[TAU], rr[TAU], ri[TAU], rz[TAU];
    auto load = [&](const void* p, T(&w)[TAU]) {
        const char* q = g.row(a, p, pl.tr, g.inb);
#pragma unroll
        for (int j = 0; j < TAU; ++j) w[j] = ld_row<R>(q, g.at(j, pl.left, g.inb));
    };
    load(a.r, rr);
    load(a.i, ri);
    load(a.x, rx);
    share_rates<G>(a, chain, s_k);
    __syncthreads();
    float k[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) k[c] = s_k[g.lc * VEC + c];
    if (pl.ragged) pad_steps<R, TAU>(mine, rr, rx);

    // the lane's steps as A[j], B[j] and composed as (P, H)
    float A[TAU][VEC], B[TAU][VEC], P[VEC], H[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) P[c] = 1.f, H[c] = 0.f;
#pragma unroll
    for (int j = 0; j < TAU; ++j) {
        bool cut = false;
        if constexpr (RESET)
            cut = j < mine && a.reset[(int64_t)g.b * a.L + pl.tw + g.rg * TAU + j] != 0;
        float x[VEC], r[VEC], i[VEC];
        R::unpack(rx[j], x);
        R::unpack(rr[j], r);
        R::unpack(ri[j], i);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float la2 = k[c] * sigmoid_f(r[c]);
            const float e = hw_exp2(la2);
            const float n = sqrt_f(one_minus_square(la2, e));
            A[j][c] = decay<RESET>(e, cut);
            B[j][c] = n * sigmoid_f(i[c]) * x[c];
            H[c] = apply<RESET>(A[j][c], H[c], B[j][c]);
            P[c] = both<RESET>(P[c], A[j][c]);
        }
        __builtin_amdgcn_sched_barrier(0);  // one step's temporaries at a time
    }
    if constexpr (GATE) load(a.z, rz);  // needed last: travels during the exchange
    // inclusive scan over the wave's time groups, then the wave's total to LDS
#pragma unroll
    for (int off = LC; off < 64; off <<= 1) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float Pu = __shfl_up(P[c], off), Hu = __shfl_up(H[c], off);
            if (g.lane >= off) {
                H[c] = apply<RESET>(P[c], Hu, H[c]);
                P[c] = both<RESET>(P[c], Pu);
            }
        }
    }
    if (g.rg == RG - 1) {
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            s_sum[g.wave][g.lc * VEC + c] = make_float2(P[c], H[c]);
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {  // exclusive
        P[c] = __shfl_up(P[c], LC);
        H[c] = __shfl_up(H[c], LC);
        if (g.rg == 0) P[c] = 1.f, H[c] = 0.f;
    }
    __syncthreads();
    if (threadIdx.x < G::CH) {  // one lane a channel: publish, look back, publish
        const Chain<G::CH> cn = chain_of<G>(a, chain);
        float bp = 1.f, bh = 0.f, hb;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 v = s_sum[w][threadIdx.x];
            bh = apply<RESET>(v.x, bh, v.y);
            bp = both<RESET>(bp, v.x);
        }
        const int64_t at = (int64_t)g.b * a.Dn + slot_channel<G>(a, chain, (int)threadIdx.x);
        if (blk > 0) {
            if (!last) cn.publish_map(blk, bp, bh);
            hb = cn.template before<RESET>(blk);
        } else {
            hb = a.h0 ? a.h0[at] : 0.f;
        }
        const float after = apply<RESET>(bp, hb, bh);
        if (!last) cn.publish_state(blk, after);
        else if (a.h_last) a.h_last[at] = after;
        s_h[threadIdx.x] = hb;
    }
    __syncthreads();
    float h[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) h[c] = s_h[g.lc * VEC + c];
    for (int w = 0; w < g.wave; ++w) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float2 v = s_sum[w][g.lc * VEC + c];
            h[c] = apply<RESET>(v.x, h[c], v.y);
        }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) h[c] = apply<RESET>(P[c], h[c], H[c]);
    if (g.live && mine > 0) {
        if (a.states && g.rg * TAU % kGatedBlock == 0) {
            const int64_t row = (int64_t)g.b * a.nstates + (pl.tw + g.rg * TAU) / kGatedBlock;
            float* st = a.states + row * a.Dn + g.ch;
#pragma unroll
            for (int c = 0; c < VEC; ++c) st[c] = h[c];
        }
        char* py = g.row(a, a.y, pl.tw, g.rowb);
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
            if (j < mine) st_row<R>(py, g.at(j, pl.left, g.rowb), R::pack(o));
        }
    }
}

// ---- backward -----------------------------------------------------------------------
// The same blocks from the end of the sequence.  Each wave starts its forward
// recurrence from the state saved before its first step, so only the message
// A_t g_t travels between waves (through LDS) and blocks.
template <class G, bool GATE, bool RESET>
__global__ void __launch_bounds__(64 * G::W, 3) gated_bwd(GatedArgs a) {
    constexpr int VEC = G::VEC, LC = G::LC, RG = G::RG, TAU = G::TAU, TW = G::TW, TB = G::TB,
                  W = G::W;
    using R = RowIo<VEC, G::BF16>;
    using T = typename R::T;
    static_assert(TW % kGatedBlock == 0, "a wave starts at a saved state");
    __shared__ float2 s_sum[W][G::CH];
    __shared__ float s_h[G::CH], s_k[G::CH];
    __shared__ float s_lam[W][G::CH];
    // h_{t-1} and the gradient arriving at h_t, a lane's own: in registers they
    // spill (4 channels x 4 steps a lane, 8 x 2048 x 1536 bf16 with gate and resets:
    // 152 us for 111, with the gate 117 for 104).
    typedef float F __attribute__((ext_vector_type(VEC)));
    __shared__ F s_hp[TAU][64 * W], s_gh[TAU][64 * W];
    const Work wk = take_work(a);
    const int64_t turn = wk.turn, blk = a.blocks - 1 - turn;  // turn 0 is the last block
    const uint32_t chain = wk.chain;
    const Place<G> pl(a, blk);
    const Lane<G> g(a, chain);
    const int64_t tw = pl.tw, tr = pl.tr;
    const int left = pl.left, mine = pl.mine(g);

    T rx[TAU], rr[TAU], ri[TAU], rz[TAU], ry[TAU];
    auto load = [&](const void* p, T(&w)[TAU], uint32_t pitch) {
        const char* q = g.row(a, p, tr, pitch);
#pragma unroll
        for (int j = 0; j < TAU; ++j) w[j] = ld_row<R>(q, g.at(j, left, pitch));
    };
    load(a.r, rr, g.inb);
    load(a.i, ri, g.inb);
    load(a.x, rx, g.inb);
    float h[VEC];
    const float* st = a.states + ((int64_t)g.b * a.nstates + tr / kGatedBlock) * a.Dn + g.ch;
#pragma unroll
    for (int c = 0; c < VEC; ++c) h[c] = st[c];
    share_rates<G>(a, chain, s_k);
    if (pl.ragged) pad_steps<R, TAU>(mine, rr, rx);
    __syncthreads();
    float k[VEC], dlam[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        k[c] = s_k[g.lc * VEC + c];
        dlam[c] = 0.f;
    }
    // forward: A, h_{t-1}
    float sr[TAU][VEC], e[TAU][VEC], A[TAU][VEC], n[TAU][VEC], si[TAU][VEC];
    float P[VEC], H[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) P[c] = 1.f, H[c] = 0.f;
#pragma unroll
    for (int j = 0; j < TAU; ++j) {
        bool cut = false;
        if constexpr (RESET)
            cut = j < mine && a.reset[(int64_t)g.b * a.L + tw + g.rg * TAU + j] != 0;
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
            A[j][c] = decay<RESET>(e[j][c], cut);
            H[c] = apply<RESET>(A[j][c], H[c], n[j][c] * si[j][c] * x[c]);
            P[c] = both<RESET>(P[c], A[j][c]);
        }
        __builtin_amdgcn_sched_barrier(0);  // one step's temporaries at a time
    }
    // Asked for here, not with the others: 8 x 2048 x 1536 bf16 102 us for 112.
    load(a.dy, ry, g.rowb);
    if constexpr (GATE) load(a.z, rz, g.inb);
    // no gradient arrives at steps past the end either
    if (pl.ragged) pad_steps<R, TAU>(mine, ry, ry);
#pragma unroll
    for (int off = LC; off < 64; off <<= 1) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float Pu = __shfl_up(P[c], off), Hu = __shfl_up(H[c], off);
            if (g.lane >= off) {
                H[c] = apply<RESET>(P[c], Hu, H[c]);
                P[c] = both<RESET>(P[c], Pu);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        float Pe = __shfl_up(P[c], LC), He = __shfl_up(H[c], LC);
        if (g.rg == 0) Pe = 1.f, He = 0.f;
        h[c] = apply<RESET>(Pe, h[c], He);
    }
    // h_{t-1} of every step, dz, and the gradient arriving at h_t from y_t
    char* oz = g.row(a, a.dz, tw, g.rowb);
#pragma unroll
    for (int j = 0; j < TAU; ++j) {
        const bool in = j < mine;
        float x[VEC], dy[VEC];
        R::unpack(rx[j], x);
        R::unpack(ry[j], dy);
        F hp, gh;
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            hp[c] = h[c];
            h[c] = apply<RESET>(A[j][c], h[c], n[j][c] * si[j][c] * x[c]);
            gh[c] = dy[c];
        }
        if constexpr (GATE) {
            float z[VEC], dz[VEC];
            R::unpack(rz[j], z);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float sz = sigmoid_f(z[c]);
                dz[c] = dy[c] * h[c] * sz * fmaf(z[c], 1.f - sz, 1.f);
                gh[c] *= z[c] * sz;
            }
            if (g.live && in) st_row<R>(oz, g.at(j, left, g.rowb), R::pack(dz));
        }
        // a padded step's own q is 0 whatever its state holds
        if (pl.ragged && !in) hp = F{}, gh = F{};
        s_hp[j][threadIdx.x] = hp;
        s_gh[j][threadIdx.x] = gh;
        __builtin_amdgcn_sched_barrier(0);
    }
    // the message to the step before the lane: c_out = P c_in + C
    float C[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) P[c] = 1.f, C[c] = 0.f;
#pragma unroll
    for (int j = TAU - 1; j >= 0; --j) {
        const F gh = s_gh[j][threadIdx.x];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            C[c] = apply<RESET>(A[j][c], gh[c] + C[c], 0.f);
            P[c] = both<RESET>(P[c], A[j][c]);
        }
    }
#pragma unroll
    for (int off = LC; off < 64; off <<= 1) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float Pd = __shfl_down(P[c], off), Cd = __shfl_down(C[c], off);
            if (g.lane + off < 64) {
                C[c] = apply<RESET>(P[c], Cd, C[c]);
                P[c] = both<RESET>(P[c], Pd);
            }
        }
    }
    if (g.rg == 0) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) s_sum[g.wave][g.lc * VEC + c] = make_float2(P[c], C[c]);
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        P[c] = __shfl_down(P[c], LC);
        C[c] = __shfl_down(C[c], LC);
        if (g.rg == RG - 1) P[c] = 1.f, C[c] = 0.f;
    }
    __syncthreads();
    if (threadIdx.x < G::CH) {  // one lane a channel: publish, look back, publish
        const Chain<G::CH> cn = chain_of<G>(a, chain);
        const bool last = blk == 0;
        float bp = 1.f, bc = 0.f, cb;
#pragma unroll
        for (int w = W - 1; w >= 0; --w) {
            const float2 q = s_sum[w][threadIdx.x];
            bc = apply<RESET>(q.x, bc, q.y);
            bp = both<RESET>(bp, q.x);
        }
        if (turn > 0) {
            if (!last) cn.publish_map(turn, bp, bc);
            cb = cn.template before<RESET>(turn);
        } else {
            cb = a.dh_last ? a.dh_last[(int64_t)g.b * a.Dn + slot_channel<G>(a, chain, (int)threadIdx.x)] : 0.f;
        }
        const float out = apply<RESET>(bp, cb, bc);
        if (!last) cn.publish_state(turn, out);
        else if (a.dh0) a.dh0[(int64_t)g.b * a.Dn + slot_channel<G>(a, chain, (int)threadIdx.x)] = out;
        s_h[threadIdx.x] = cb;
    }
    __syncthreads();
    float m[VEC];  // the message arriving from the step after the lane's last
#pragma unroll
    for (int c = 0; c < VEC; ++c) m[c] = s_h[g.lc * VEC + c];
    for (int w = W - 1; w > g.wave; --w) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float2 q = s_sum[w][g.lc * VEC + c];
            m[c] = apply<RESET>(q.x, m[c], q.y);
        }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) m[c] = apply<RESET>(P[c], m[c], C[c]);
    char *ox = g.row(a, a.dx, tw, g.rowb), *orr = g.row(a, a.dr, tw, g.rowb),
         *oi = g.row(a, a.di, tw, g.rowb);
#pragma unroll
    for (int j = TAU - 1; j >= 0; --j) {
        const bool in = j < mine;
        float x[VEC], dx[VEC], dr[VEC], di[VEC];
        R::unpack(rx[j], x);
        const F gh = s_gh[j][threadIdx.x], hp = s_hp[j][threadIdx.x];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float gt = gh[c] + m[c];  // dL/dh_t
            m[c] = apply<RESET>(A[j][c], gt, 0.f);
            const float s = si[j][c], la = k[c] * kLn2 * sr[j][c];
            const float ratio = n[j][c] > 0.f ? la * hw_rcp(n[j][c]) : 0.f;
            const float keep = apply<RESET>(A[j][c], hp[c], 0.f) * la;
            const float q = gt * fmaf(-s * x[c] * e[j][c], e[j][c] * ratio, keep);
            dx[c] = gt * n[j][c] * s;
            di[c] = dx[c] * x[c] * (1.f - s);
            dr[c] = q * (1.f - sr[j][c]);
            dlam[c] += q;
        }
        if (g.live && in) {
            const uint32_t o = g.at(j, left, g.rowb);
            st_row<R>(ox, o, R::pack(dx));
            st_row<R>(orr, o, R::pack(dr));
            st_row<R>(oi, o, R::pack(di));
        }
        __builtin_amdgcn_sched_barrier(0);
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
    if (threadIdx.x < G::CH && (int)(chain % tiles_of<G>(a)) * G::CH +
                                       (int)threadIdx.x / VEC * VEC < a.Dn) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += s_lam[w][threadIdx.x];
        a.part[((int64_t)g.b * a.blocks + blk) * a.Dn + slot_channel<G>(a, chain, (int)threadIdx.x)] = v;
    }
}

// dlam[d] = sigmoid/softplus(lam) * sum of the partials over `rows`: 16 waves
// take equal ranges of rows for 64 channels, joined in order.
constexpr int kLamWaves = 16;
__global__ void __launch_bounds__(64 * kLamWaves) gated_dlam(GatedArgs a, int64_t rows) {
    __shared__ float s_v[kLamWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int d = blockIdx.x * 64 + lane;
    const int64_t r0 = rows * wave / kLamWaves, r1 = rows * (wave + 1) / kLamWaves;
    float v = 0.f;
    if (d < a.Dn) {
        int64_t i = r0;
        for (; i + 8 <= r1; i += 8) {
            float w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = a.part[(i + u) * a.Dn + d];
#pragma unroll
            for (int u = 0; u < 8; ++u) v += w[u];
        }
        for (; i < r1; ++i) v += a.part[i * a.Dn + d];
    }
    s_v[wave][lane] = v;
    __syncthreads();
    if (wave != 0 || d >= a.Dn) return;
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kLamWaves; ++w) v += s_v[w][lane];
    a.dlam[d] = v * sigmoid_over_softplus(a.lam[d]);
}

// ---- one step ------------------------------------------------------------------------
// A thread takes VEC channels of BR batch rows, so that the rate's logarithm
// is taken once for all of them and their loads travel together.  Bound by its
// bytes, h read and written and one row of each input, and below some ten
// megabytes by the launch: 256 x 5120 bf16 moves 23.6 MB in 8.3 us (2.8 TB/s),
// of which about 3 us are a launch that does nothing.
template <int VEC, int BR, bool BF16>
__global__ void __launch_bounds__(256) gated_step(GatedArgs a) {
    using R = RowIo<VEC, BF16>;
    using T = typename R::T;
    typedef float F __attribute__((ext_vector_type(VEC)));
    const int vecs = a.Dn / VEC, rows = (a.batch + BR - 1) / BR;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row0 = (int)(t / (uint32_t)vecs) * BR, v = (int)(t % (uint32_t)vecs);
    if (t >= (int64_t)rows * vecs) return;
    F h[BR];
    T x[BR], r[BR], i[BR], z[BR];
#pragma unroll
    for (int k = 0; k < BR; ++k) {
        const int64_t row = min(row0 + k, a.batch - 1);
        h[k] = reinterpret_cast<const F*>(a.h_last)[row * vecs + v];
        auto in = [&](const void* p) {
            return *reinterpret_cast<const typename R::M*>(static_cast<const typename R::E*>(p) +
                                                           row * a.ld + v * VEC);
        };
        r[k] = in(a.r);
        i[k] = in(a.i);
        x[k] = in(a.x);
        if (a.z) z[k] = in(a.z);
    }
    float rate[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c)
        rate[c] = -a.sharp * kLog2e * softplus_rel(a.lam[v * VEC + c]);
#pragma unroll
    for (int k = 0; k < BR; ++k) {
        if (row0 + k >= a.batch) break;
        const int64_t at = (int64_t)(row0 + k) * vecs + v;
        float xf[VEC], rf[VEC], gf[VEC], o[VEC];
        R::unpack(x[k], xf);
        R::unpack(r[k], rf);
        R::unpack(i[k], gf);
        F hn;
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float la2 = rate[c] * sigmoid_f(rf[c]);
            const float e = hw_exp2(la2);
            const float n = sqrt_f(one_minus_square(la2, e));
            o[c] = fmaf(e, h[k][c], n * sigmoid_f(gf[c]) * xf[c]);
            hn[c] = o[c];
        }
        reinterpret_cast<F*>(a.h_last)[at] = hn;
        if (a.z) {
            float zf[VEC];
            R::unpack(z[k], zf);
#pragma unroll
            for (int c = 0; c < VEC; ++c) o[c] *= silu_f(zf[c]);
        }
        static_cast<T*>(a.y)[at] = R::pack(o);
    }
}

// ---- variants -------------------------------------------------------------------------
// The lanes across channels take a line of 128 bytes of bf16 in each row.  As
// many steps a lane as registers hold (3 waves a SIMD; without resets nothing
// spills, with them 36 to 57 scalar registers of the forward, and 5 vector
// registers of the fp32 backward with the gate), since each lane's map costs a
// scan over the lanes: with 2 channels a lane instead of 4 the forward has half as
// many lanes to scan over.  Forward at 8 x 2048 x 1536 bf16 with the gate and at
// 131072 x 1536 without, in us: 58 and 333; 4 channels x 8 steps a lane 60 and 349
// (with 2 waves along time 59 and 497, with 8 70 and 380), 1 x 32 73 and 331, 2 x 8
// 56 and 391 (shorter blocks make the chain of messages longer).  Backward at the
// first: 100; 4 channels x 4 steps a lane 107 (with 2 waves along time 110, with 8
// 130), 1 x 16 110.
template <bool BF16>
using Fwd = Geo<2, 32, 16, 4, BF16>;
template <bool BF16>
using Bwd = Geo<2, 32, 8, 4, BF16>;
// fewer than four channels
template <bool BF16>
using FwdOne = Geo<1, 4, 2, 4, BF16>;
template <bool BF16>
using BwdOne = Geo<1, 4, 1, 4, BF16>;

// The sizes that a launch and its workspace go by.
struct Cut {
    int ch, tb, w;
    int64_t chains, blocks;
};
template <class G>
Cut cut_of(int batch, int64_t L, int Dn) {
    return Cut{G::CH, G::TB, G::W, (int64_t)((Dn + G::CH - 1) / G::CH) * batch,
               (L + G::TB - 1) / G::TB};
}
Cut fwd_cut(int batch, int64_t L, int Dn, bool bf16) {
    if (Dn < 4) return cut_of<FwdOne<true>>(batch, L, Dn);
    return bf16 ? cut_of<Fwd<true>>(batch, L, Dn) : cut_of<Fwd<false>>(batch, L, Dn);
}
Cut bwd_cut(int batch, int64_t L, int Dn, bool bf16) {
    if (Dn < 4) return cut_of<BwdOne<true>>(batch, L, Dn);
    return bf16 ? cut_of<Bwd<true>>(batch, L, Dn) : cut_of<Bwd<false>>(batch, L, Dn);
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Words between blocks: [tickets][room in front][words]; nothing for one block.
struct Ws {
    size_t word, words, total;
};
Ws ws_of(const Cut& c) {
    Ws w{};
    if (c.blocks < 2) return w;
    w.words = (size_t)c.chains * (size_t)c.blocks * c.ch;
    const size_t front = (size_t)kWindow * c.ch;  // read, never taken (Chain::before)
    w.word = up256((size_t)c.chains * kTicketStride * 4) + up256(front * 8);
    w.total = w.word + up256(w.words * 8);
    return w;
}

hipError_t prepare(GatedArgs& a, const Cut& c, void* workspace, hipStream_t s) {
    a.blocks = c.blocks;
    a.chains = (uint32_t)c.chains;
    if (c.blocks < 2) return hipSuccess;
    const Ws w = ws_of(c);
    char* ws = static_cast<char*>(workspace);
    a.ticket = reinterpret_cast<uint32_t*>(ws);
    a.word = reinterpret_cast<uint64_t*>(ws + w.word);
    ProfScope ps(s, kPhasePrep);
    const size_t n = (w.words + 255) / 256;
    hipLaunchKernelGGL(gated_prepare, dim3((unsigned)(n < 2048 ? n : 2048)), dim3(256), 0, s, a,
                       (int64_t)w.words);
    return hipGetLastError();
}

#define MS_GATED_VARIANT_(kernel, ...)                                                           \
    do {                                                                                         \
        if (a.z && a.reset) hipLaunchKernelGGL((kernel<__VA_ARGS__, true, true>), grid, blk, 0, s, a); \
        else if (a.z) hipLaunchKernelGGL((kernel<__VA_ARGS__, true, false>), grid, blk, 0, s, a);      \
        else if (a.reset) hipLaunchKernelGGL((kernel<__VA_ARGS__, false, true>), grid, blk, 0, s, a);  \
        else hipLaunchKernelGGL((kernel<__VA_ARGS__, false, false>), grid, blk, 0, s, a);              \
    } while (0)

}  // namespace

int64_t gated_workgroups(int batch, int64_t L, int Dn, bool bf16) {
    const Cut f = fwd_cut(batch, L, Dn, bf16), b = bwd_cut(batch, L, Dn, bf16);
    const double n = (double)f.chains * (double)f.blocks, m = (double)b.chains * (double)b.blocks;
    return (int64_t)(n > m ? n : m);
}

// An odd channel count: one channel belongs to two lanes, maybe of two
// workgroups, and where h_last lies over h0 one may store it before the other
// has read it.  Then h0 is copied first.
static size_t start_bytes(int batch, int Dn) {
    return Dn > 4 && Dn % 2 ? up256((size_t)batch * (size_t)Dn * 4) : 0;
}

size_t gated_fwd_ws(int batch, int64_t L, int Dn, bool bf16) {
    return ws_of(fwd_cut(batch, L, Dn, bf16)).total + start_bytes(batch, Dn);
}

// The backward's partial sums of dlam follow its words.
size_t gated_bwd_ws(int batch, int64_t L, int Dn, bool bf16) {
    const Cut c = bwd_cut(batch, L, Dn, bf16);
    return ws_of(c).total + up256((size_t)batch * (size_t)c.blocks * (size_t)Dn * 4);
}

hipError_t launch_gated_fwd(GatedArgs a, bool bf16, void* workspace, hipStream_t s) {
    const Cut c = fwd_cut(a.batch, a.L, a.Dn, bf16);
    const hipError_t e = prepare(a, c, workspace, s);
    if (e != hipSuccess) return e;
    if (a.h0 && a.h0 == a.h_last && start_bytes(a.batch, a.Dn)) {
        float* start = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws_of(c).total);
        const int64_t n = (int64_t)a.batch * a.Dn, g = (n + 255) / 256;
        ProfScope ps(s, kPhasePrep);
        hipLaunchKernelGGL(gated_copy, dim3((unsigned)(g < 2048 ? g : 2048)), dim3(256), 0, s,
                           a.h0, start, n);
        a.h0 = start;
    }
    ProfScope ps(s, kPhaseMain);
    const dim3 grid((unsigned)(c.chains * c.blocks)), blk(64 * c.w);
    if (a.Dn >= 4) {
        if (bf16) MS_GATED_VARIANT_(gated_fwd, Fwd<true>);
        else MS_GATED_VARIANT_(gated_fwd, Fwd<false>);
    } else {
        if (bf16) MS_GATED_VARIANT_(gated_fwd, FwdOne<true>);
        else MS_GATED_VARIANT_(gated_fwd, FwdOne<false>);
    }
    return hipGetLastError();
}

hipError_t launch_gated_bwd(GatedArgs a, bool bf16, void* workspace, hipStream_t s) {
    const Cut c = bwd_cut(a.batch, a.L, a.Dn, bf16);
    hipError_t e = prepare(a, c, workspace, s);
    if (e != hipSuccess) return e;
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws_of(c).total);
    {
        ProfScope ps(s, kPhaseMain);
        const dim3 grid((unsigned)(c.chains * c.blocks)), blk(64 * c.w);
        if (a.Dn >= 4) {
            if (bf16) MS_GATED_VARIANT_(gated_bwd, Bwd<true>);
            else MS_GATED_VARIANT_(gated_bwd, Bwd<false>);
        } else {
            if (bf16) MS_GATED_VARIANT_(gated_bwd, BwdOne<true>);
            else MS_GATED_VARIANT_(gated_bwd, BwdOne<false>);
        }
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ProfScope ps(s, kPhaseReduce);
    hipLaunchKernelGGL(gated_dlam, dim3((a.Dn + 63) / 64), dim3(64 * kLamWaves), 0, s, a,
                       (int64_t)a.batch * a.blocks);
    return hipGetLastError();
}

// Two batch rows a thread where that leaves the chip half full of threads or
// more (256 x 5120 bf16: 8.3 us, one row 9.1, four 8.6, eight 9.0).
static int step_rows(const GatedArgs& a) {
    return a.Dn % 4 == 0 && (int64_t)a.batch * (a.Dn / 4) >= 256 * 1024 ? 2 : 1;
}

int64_t gated_step_workgroups(const GatedArgs& a) {
    const int br = step_rows(a), vecs = a.Dn % 4 ? a.Dn : a.Dn / 4;
    return ((int64_t)((a.batch + br - 1) / br) * vecs + 255) / 256;
}

hipError_t launch_gated_step(const GatedArgs& a, bool bf16, hipStream_t s) {
    ProfScope ps(s, kPhaseStep);
    const dim3 grid((unsigned)gated_step_workgroups(a)), blk(256);
    if (a.Dn % 4) {
        if (bf16) hipLaunchKernelGGL((gated_step<1, 1, true>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((gated_step<1, 1, false>), grid, blk, 0, s, a);
    } else if (step_rows(a) == 2) {
        if (bf16) hipLaunchKernelGGL((gated_step<4, 2, true>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((gated_step<4, 2, false>), grid, blk, 0, s, a);
    } else {
        if (bf16) hipLaunchKernelGGL((gated_step<4, 1, true>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((gated_step<4, 1, false>), grid, blk, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace msscan
