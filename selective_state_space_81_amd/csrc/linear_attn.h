// linear_attn.h -- what the kernels of the linear attention share: operand
// fragments of the matrix instructions, tiles of tokens in LDS, and the decays
// inside a block of tokens.  Included only by linear_attn*.hip.
//
// Notation: a block is kBlock tokens of one head.  With G_i the sum of the log
// decays up to token i of the block (in base 2), and a document starting at
// start_i <= i,
//   o_i    = scale sum_{start_i <= j <= i} 2^(G_i - G_j) (q_i . k_j) v_j
//            + scale 2^G_i S^T q_i        (S before the block; no start up to i)
//   S_next = 2^G_last S + sum_j 2^(G_last - G_j) k_j v_j^T     (of the last document)
#pragma once

#include <type_traits>

#include "device_common.h"
#include "dpp64.h"
#include "lm_internal.h"

namespace msscan {
namespace attn {

using namespace dev;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f8 __attribute__((ext_vector_type(8)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef u4 u4_align2 __attribute__((aligned(2)));
typedef u4 u4_align4 __attribute__((aligned(4)));
typedef f8 f8_align16 __attribute__((aligned(16)));
typedef u2 u2_align2 __attribute__((aligned(2)));
typedef f4 f4_align4 __attribute__((aligned(4)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;

// A barrier for what waves share in LDS.  __syncthreads also waits for every
// load and store of global memory under way, the next block's inputs among them.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ---- operands of the matrix instructions ---------------------------------------
//
// D = A B over 32 of the summed index.  Lane l = 16 g + s holds row s of A (or
// column s of B), entries 8 g .. 8 g + 7 of the summed index, and of D column
// s, rows 4 g .. 4 g + 3.  In bf16 that is one 16x16x32 instruction; in fp32
// eight 16x16x4 ones, the e-th of which takes entry e of every lane: the order
// of a sum does not matter to which operands meet.
template <bool BF16>
struct Io;
template <>
struct Io<true> {
    typedef uint16_t E;
    typedef b8 Frag;
    typedef b4 Half;
    static constexpr int kBlock = kAttnBlockBf16;
    static constexpr int kPad = 8;  // of a row of LDS: rows of 16 lanes fall on all banks
    static constexpr int kParts = 3;
};
template <>
struct Io<false> {
    typedef float E;
    typedef f8 Frag;
    typedef f4 Half;
    static constexpr int kBlock = kAttnBlockF32;
    static constexpr int kPad = 4;
    static constexpr int kParts = 1;
};

__device__ __forceinline__ f4 mma(b8 a, b8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mma(f8 a, f8 b, f4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// fp32 values as an operand.  round() keeps 8 bits of them in bf16: what it is
// used for (scores, the state that a query meets; in the gradient the scores and
// their gradients, and R for dv) ends in a bf16 output and adds as much error as
// that output's own rounding.  Parts keeps all 24 bits, as a sum of three bf16
// numbers, for what ends in fp32 (states, gradients of decays): two would leave
// 3e-6 of a state, three leave fp32's own error.  The parts of an infinite value
// sum to NaN.  That is let be: it is met in gradients alone, where an infinite
// state leaves nothing finite, and a second way through them for it cost 6 of 322
// us of a training pass where all is finite.
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack(float lo, float hi) {  // one conversion for both
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{lo, hi}), b2));
}
__device__ __forceinline__ b8 round(f8 x, b8) {
    return __builtin_bit_cast(b8, u4{pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]),
                                     pack(x[6], x[7])});
}
__device__ __forceinline__ f8 round(f8 x, f8) { return x; }
__device__ __forceinline__ f8 widen(b8 x) {
    f8 y;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (float)x[e];
    return y;
}
__device__ __forceinline__ f8 widen(f8 x) { return x; }

template <bool BF16>
struct Parts {
    typename Io<BF16>::Frag p[Io<BF16>::kParts];
    __device__ __forceinline__ explicit Parts(f8 x) {
        if constexpr (BF16) {
            u4 part[3];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo = x[2 * e], hi = x[2 * e + 1];
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    part[n][e] = pack(lo, hi);
                    lo -= __uint_as_float(part[n][e] << 16);
                    hi -= __uint_as_float(part[n][e] & 0xffff0000u);
                }
            }
#pragma unroll
            for (int n = 0; n < 3; ++n) p[n] = __builtin_bit_cast(b8, part[n]);
        } else {
            p[0] = x;
        }
    }
    __device__ __forceinline__ f4 times(typename Io<BF16>::Frag b, f4 c) const {
#pragma unroll
        for (int n = Io<BF16>::kParts - 1; n >= 0; --n) c = mma(p[n], b, c);
        return c;
    }
};

// A lane's 8 entries of an operand from a tile in LDS, rows of LD values:
// along(): operand index = tile row, summed index along the row;
// across(): operand index = tile column, summed index down the rows (in bf16 by
// the transposing read: 16 lanes read 4 rows of 16 columns, a lane gets a column).
template <int LD>
__device__ __forceinline__ b8 along(const uint16_t* tile, int row0, int k0) {
    const int l = threadIdx.x & 63;
    return *reinterpret_cast<const b8*>(tile + (row0 + (l & 15)) * LD + k0 + (l >> 4) * 8);
}
template <int LD>
__device__ __forceinline__ f8 along(const float* tile, int row0, int k0) {
    const int l = threadIdx.x & 63;
    const float* p = tile + (row0 + (l & 15)) * LD + k0 + (l >> 4) * 8;
    const f4 a = *reinterpret_cast<const f4*>(p), b = *reinterpret_cast<const f4*>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int LD>
__device__ __forceinline__ b8 across(const uint16_t* tile, int k0, int col0) {
    typedef __attribute__((address_space(3))) s4* Lds;
    const int l = threadIdx.x & 63, g = l >> 4, s = l & 15;
    const uint16_t* p = tile + (k0 + g * 8 + (s >> 2)) * LD + col0 + (s & 3) * 4;
    const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p);
    const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * LD));
    return __builtin_bit_cast(b8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int LD>
__device__ __forceinline__ f8 across(const float* tile, int k0, int col0) {
    const int l = threadIdx.x & 63;
    const float* p = tile + (k0 + (l >> 4) * 8) * LD + col0 + (l & 15);
    f8 y;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = p[e * LD];
    return y;
}
// The same for a summed index that is taken 4 + 4 from two blocks of 16, as two
// tiles of D hold them: rows k0 + 4 g .. and k0 + 16 + 4 g ..
template <int LD>
__device__ __forceinline__ b8 across_pair(const uint16_t* tile, int k0, int col0) {
    typedef __attribute__((address_space(3))) s4* Lds;
    const int l = threadIdx.x & 63, g = l >> 4, s = l & 15;
    const uint16_t* p = tile + (k0 + g * 4 + (s >> 2)) * LD + col0 + (s & 3) * 4;
    const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p);
    const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 16 * LD));
    return __builtin_bit_cast(b8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int LD>
__device__ __forceinline__ f8 across_pair(const float* tile, int k0, int col0) {
    const int l = threadIdx.x & 63;
    const float* p = tile + (k0 + (l >> 4) * 4) * LD + col0 + (l & 15);
    f8 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        y[e] = p[e * LD];
        y[4 + e] = p[(16 + e) * LD];
    }
    return y;
}

__device__ __forceinline__ void put4(uint16_t* p, f4 x) {
    *reinterpret_cast<u2*>(p) = u2{pack(x[0], x[1]), pack(x[2], x[3])};
}
__device__ __forceinline__ void put4(float* p, f4 x) { *reinterpret_cast<f4*>(p) = x; }
__device__ __forceinline__ void put8(uint16_t* p, b8 x) { *reinterpret_cast<b8*>(p) = x; }
__device__ __forceinline__ void put8(float* p, f8 x) { *reinterpret_cast<f8_align16*>(p) = x; }
__device__ __forceinline__ float get(const uint16_t* p) {
    return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ f4 get4(const uint16_t* p) {
    const b4 x = *reinterpret_cast<const b4*>(p);
    f4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (float)x[e];
    return y;
}
__device__ __forceinline__ f4 get4(const float* p) { return *reinterpret_cast<const f4*>(p); }

// Four values of a row of n from place i on, where they are in it (WHOLE: all of
// them or none).
template <bool WHOLE, class E>
__device__ __forceinline__ void store4(E* row, int i, int n, f4 x) {
    if (WHOLE ? i < n : i + 4 <= n) {
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<u2_align2*>(row + i) = u2{pack(x[0], x[1]), pack(x[2], x[3])};
        else
            *reinterpret_cast<f4_align4*>(row + i) = x;
    } else if (!WHOLE) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (i + e < n) st<sizeof(E) == 2>(row, i + e, x[e]);
    }
}

// ---- tiles of tokens --------------------------------------------------------------

// The eight values of a vector moved down by s places, whose last s are lost.
template <bool BF16>
__device__ __forceinline__ void move_down(uint32_t (&x)[BF16 ? 4 : 8], int s) {
    constexpr int kWords = BF16 ? 4 : 8;
    if constexpr (BF16) {
        const bool half = s & 1;
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            x[w] = half ? x[w] >> 16 | (w + 1 < kWords ? x[w + 1] << 16 : 0) : x[w];
        s >>= 1;
    }
#pragma unroll
    for (int d = 1; d < kWords; d *= 2) {
        const bool on = s & d;
#pragma unroll
        for (int w = 0; w < kWords; ++w) x[w] = on ? (w + d < kWords ? x[w + d] : 0) : x[w];
    }
}

// kBlock rows of W values (n of them there), from global memory through
// registers to LDS, zeros beyond the rows and columns that there are.  Rows lie
// less than 2^22 values apart, so 32 bits hold a place in a block.
// Loads need no branch, which would wait for each: they ask for whole vectors
// that are there, and nothing waits for them until store(), which moves a row's
// last values to where they belong (WHOLE: n is a multiple of 8, and none has
// to) and clears what lies beyond.  Rows of less than 8 values are the exception.
template <bool BF16, int W, bool WHOLE, int THREADS = kThreads>
struct Tile {
    typedef typename Io<BF16>::E E;
    static constexpr int kRows = Io<BF16>::kBlock;
    static constexpr int kLd = W + Io<BF16>::kPad;
    static constexpr int kVecs = W / 8;  // of 8 values, in a row
    static constexpr bool kFew = kRows * kVecs < THREADS;  // not a vector for every thread
    static constexpr int kMine = kFew ? 1 : kRows * kVecs / THREADS;
    static constexpr int kStep = THREADS / kVecs;  // rows between a thread's vectors
    static constexpr int kWords = BF16 ? 4 : 8;    // 32-bit words of 8 values
    static constexpr int kSize = kRows * kLd;      // in LDS, values
    static_assert((kFew || kRows * kVecs % THREADS == 0) && THREADS % kVecs == 0,
                  "whole rounds of the threads, which keep their columns");
    uint32_t r[kMine][kWords];

    __device__ __forceinline__ void vector(int m, const E* p) {
        typedef typename std::conditional<BF16, u4_align2, u4_align4>::type V;
#pragma unroll
        for (int h = 0; h < kWords / 4; ++h) {
            const u4 x = *reinterpret_cast<const V*>(p + h * (BF16 ? 8 : 4));
#pragma unroll
            for (int w = 0; w < 4; ++w) r[m][h * 4 + w] = x[w];
        }
    }
    __device__ __forceinline__ void load(const E* base, int ld, int rows, int n) {
        const int last = (rows < kRows ? rows : kRows) - 1;
        const int row = threadIdx.x / kVecs, c = threadIdx.x % kVecs * 8;
        if (WHOLE || n >= 8) {
            if (!kFew && rows >= kRows) {
                const uint32_t at = row * ld + min(c, n - 8);
#pragma unroll
                for (int m = 0; m < kMine; ++m) vector(m, base + m * kStep * ld + at);
            } else {
#pragma unroll
                for (int m = 0; m < kMine; ++m)
                    vector(m, base + (uint32_t)(min(row + m * kStep, last) * ld +
                                                min(c, n - 8)));
            }
            return;
        }
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const E* p = base + (uint32_t)(min(row + m * kStep, last) * ld);
#pragma unroll
            for (int w = 0; w < kWords; ++w) r[m][w] = 0;
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) {
                    if constexpr (BF16)
                        r[m][e / 2] |= (uint32_t)p[e] << (e % 2 * 16);
                    else
                        r[m][e] = __float_as_uint(p[e]);
                }
        }
    }
    // To LDS; whether something was infinite or NaN.
    __device__ __forceinline__ bool store(E* tile, int rows, int n) {
        uint32_t bad = 0;
        const int row = threadIdx.x / kVecs, c = threadIdx.x % kVecs * 8;
        if (kFew && row >= kRows) return false;
        if (!WHOLE && n >= 8) {
            const int s = min(max(c + 8 - n, 0), 8);
#pragma unroll
            for (int m = 0; m < kMine; ++m) move_down<BF16>(r[m], s);
        }
        if (rows < kRows || n < W) {
#pragma unroll
            for (int m = 0; m < kMine; ++m)
                if (!(row + m * kStep < rows && c < n))
#pragma unroll
                    for (int w = 0; w < kWords; ++w) r[m][w] = 0;
        }
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
#pragma unroll
            for (int h = 0; h < kWords / 4; ++h)
                *reinterpret_cast<u4*>(tile + (row + m * kStep) * kLd + c + h * 4) =
                    u4{r[m][h * 4], r[m][h * 4 + 1], r[m][h * 4 + 2], r[m][h * 4 + 3]};
            // an exponent of all ones, plus one, carries into the sign's place
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                bad |= BF16 ? (r[m][w] & 0x7f807f80u) + 0x00800080u
                            : (r[m][w] & 0x7f800000u) + 0x00800000u;
        }
        return (bad & (BF16 ? 0x80008000u : 0x80000000u)) != 0;
    }
};

// 16 rows of W values as operands (along(), by lane), from global memory
// straight into registers: what only one wave reads needs no LDS.
template <bool BF16, int W, bool WHOLE>
struct Rows {
    typedef typename Io<BF16>::E E;
    typedef typename Io<BF16>::Frag Frag;
    static constexpr int kSteps = W / 32;
    static constexpr int kWords = BF16 ? 4 : 8;
    uint32_t r[kSteps][kWords];

    __device__ __forceinline__ void load(const E* base, int ld, int row0, int rows, int n) {
        const int l = threadIdx.x & 63;
        const int row = min(row0 + (l & 15), rows - 1) * ld;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int c = s * 32 + (l >> 4) * 8;
            typedef typename std::conditional<BF16, u4_align2, u4_align4>::type V;
            if (WHOLE || n >= 8) {
                const E* p = base + (uint32_t)(row + min(c, n - 8));
#pragma unroll
                for (int h = 0; h < kWords / 4; ++h) {
                    const u4 x = *reinterpret_cast<const V*>(p + h * (BF16 ? 8 : 4));
#pragma unroll
                    for (int w = 0; w < 4; ++w) r[s][h * 4 + w] = x[w];
                }
            } else {
                const E* p = base + (uint32_t)row;
#pragma unroll
                for (int w = 0; w < kWords; ++w) r[s][w] = 0;
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < n) {
                        if constexpr (BF16)
                            r[s][e / 2] |= (uint32_t)p[e] << (e % 2 * 16);
                        else
                            r[s][e] = __float_as_uint(p[e]);
                    }
            }
        }
    }
    __device__ __forceinline__ Frag operand(int s, int n) const {
        typedef uint32_t U __attribute__((ext_vector_type(kWords)));
        const int c = s * 32 + (int)((threadIdx.x & 63) >> 4) * 8;
        uint32_t y[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w) y[w] = r[s][w];
        if (!WHOLE && n >= 8) move_down<BF16>(y, min(max(c + 8 - n, 0), 8));
        U x;
#pragma unroll
        for (int w = 0; w < kWords; ++w) x[w] = c < n ? y[w] : 0;
        return __builtin_bit_cast(Frag, x);
    }
};

// ---- decays of a block ---------------------------------------------------------------

// x where `in`, else 0.  What computes x is kept out of the compiler's sight: a
// branch around each exponential costs more than the exponentials.
__device__ __forceinline__ float only(bool in, float x) {
    asm volatile("" : "+v"(x));
    return in ? x : 0.f;
}

// Decay from token j to token i (of whatever document), from the sums of log decays.
__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
    return hw_exp2((hi_i - hi_j) + (lo_i - lo_j));
}

// Sums of log decays in two floats each: they reach hundreds inside a block,
// and the decay between neighbours needs the difference to 2^-24.  They run from
// the block's start, or from the document's where that lies in the block.
template <int N>
struct Decays {
    __align__(16) float hi[N];
    __align__(16) float lo[N];
    float first[N];  // 2^G_i, from the block's start to token i; 0 behind a document's start
    float last[N];   // 2^(G_last - G_i), from token i to the block's end; 0 before a start
    int start[N];    // where i's document starts in the block, or -1 before it
    float whole;     // 2^G_last; 0 where a document starts in the block

    // By one wave, lane i for token i (g: its log decay; cut: it starts a
    // document).
    __device__ __forceinline__ void make(float g, bool cut) {
        const int i = threadIdx.x & 63;
        double G = cut || i >= N ? 0.0 : (double)g * 1.4426950408889634;
        const uint64_t cuts = __ballot(cut && i < N);
        const uint64_t upto = cuts & (~0ull >> (63 - i));
        const int s = upto ? 63 - __builtin_clzll(upto) : -1;
        // Sums begin anew with a document: differences across a start are never
        // used, and a decay that is no number stays in its document.
        G = cuts ? scan64_from(G, s) : scan64(G);
        const float h = (float)G, l = (float)(G - (double)h);
        const double end = lane64(G, N - 1);
        const int send = cuts ? 63 - __builtin_clzll(cuts) : -1;
        if (i < N) {
            hi[i] = h;
            lo[i] = l;
            first[i] = s < 0 ? hw_exp2(h) * fmaf(l, kLn2, 1.f) : 0.f;
            const double d = end - G;
            const float dh = (float)d;
            last[i] = i >= send ? hw_exp2(dh) * fmaf((float)(d - (double)dh), kLn2, 1.f) : 0.f;
            start[i] = s;
            if (i == N - 1) whole = s < 0 ? first[i] : 0.f;
        }
    }
    __device__ __forceinline__ bool cut() const { return start[N - 1] >= 0; }
};

// A decay that is 0 in fp32 starts a document.
constexpr float kNoDecay = -104.f;

// Place of the log decay of (batch row, token, head).
__device__ __forceinline__ float log_decay(const AttnArgs& a, int64_t row, int h) {
    return a.fixed ? a.g[h] : a.g[row * a.H + h];
}

// A lane's token of a block: its log decay and whether a document starts, asked
// for ahead and looked at only when the block's turn comes.
struct Token {
    float g;
    uint32_t reset;
    __device__ __forceinline__ void load(const AttnArgs& a, int64_t row0, int rows, int h, int n) {
        const int i = min((int)(threadIdx.x & 63), min(rows, n) - 1);
        g = log_decay(a, row0 + i, h);
        reset = 0;
        if (a.reset) reset = a.reset[row0 + i];
    }
    // behind the last token the state stays as it is
    __device__ __forceinline__ void settle(int rows) {
        const bool in = (int)(threadIdx.x & 63) < rows;
        g = in ? g : 0.f;
        reset = in && (reset || g < kNoDecay);
    }
};

}  // namespace attn
}  // namespace msscan
