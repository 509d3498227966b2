// embed.hip -- embedding lookup with scaling (ms_embed_fwd) and its gradient
// by sorted tokens (ms_embed_bwd):
//
//   out[i][:] = scale * weight[ids[i]][:]
//   dweight[v][:] = scale * sum over i with ids[i] == v, in order of i, of dy[i][:]
//
// Both move rows and do next to no arithmetic: they are bound by memory.  The
// gradient sorts (id, position) pairs by id, stably, so that equal tokens are
// neighbours in the order they came; each workgroup then sums a fixed number
// of sorted rows, and a run of one token that crosses workgroups is joined
// from its pieces in order.  No floating-point atomics: results repeat bit for
// bit, and a token that fills much of the batch costs no more than others.
//
// Measured (5.6 TB/s is what a copy reaches).  Lookup of 16384 rows of 768 bf16
// in a table of 50280: 50 MB in 8.1 us (rows asked for twice come from the
// cache).  Gradient of the same: 43 us, of which 20 sort (two passes of 3.5 + 6.6, bound
// by their chain of dependent steps), 17 sum and write the table (102 MB, 5.9
// TB/s) and 6 join.  131072 x 2048 fp32: 603 us, the sum 575 of them (3.2 GB,
// 5.6 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "lm_internal.h"
#include "msscan_internal.h"

namespace msscan {
namespace {

using namespace dev;

// 16 bytes of a row (8 bf16 or 4 fp32 values); rows need no alignment beyond
// their element's.
template <bool BF16, int VEC>
struct Vec;
template <>
struct Vec<true, 8> {
    typedef uint16_t E;
    typedef uint32_t T __attribute__((ext_vector_type(4)));
    typedef T M __attribute__((aligned(2)));
    static __device__ __forceinline__ void unpack(T w, float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ T pack(const float (&v)[8]) {
        T w;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = (uint32_t)f32_to_bf16_rne(v[2 * k]) |
                   ((uint32_t)f32_to_bf16_rne(v[2 * k + 1]) << 16);
        return w;
    }
};
template <>
struct Vec<true, 1> {
    typedef uint16_t E;
    typedef uint16_t T;
    typedef T M;
    static __device__ __forceinline__ void unpack(T w, float (&v)[1]) {
        v[0] = __uint_as_float((uint32_t)w << 16);
    }
    static __device__ __forceinline__ T pack(const float (&v)[1]) { return f32_to_bf16_rne(v[0]); }
};
template <>
struct Vec<false, 4> {
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
struct Vec<false, 1> {
    typedef float E;
    typedef float T;
    typedef T M;
    static __device__ __forceinline__ void unpack(T w, float (&v)[1]) { v[0] = w; }
    static __device__ __forceinline__ T pack(const float (&v)[1]) { return v[0]; }
};
template <class V>
__device__ __forceinline__ typename V::T ldv(const typename V::E* p) {
    return *reinterpret_cast<const typename V::M*>(p);
}
template <class V>
__device__ __forceinline__ void stv(typename V::E* p, typename V::T v) {
    *reinterpret_cast<typename V::M*>(p) = v;
}

// A VEC-wide store in the gradient's own type: bf16 values as 16, 8 or 2
// bytes, fp32 values as 16-byte pieces.
template <int VEC, bool BF16>
__device__ __forceinline__ void store_grad(void* base, int64_t off, const float (&v)[VEC]) {
    if constexpr (BF16 && VEC == 4) {
        typedef uint32_t T __attribute__((ext_vector_type(2)));
        typedef T M __attribute__((aligned(2)));
        const T w = {(uint32_t)f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16),
                     (uint32_t)f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16)};
        *reinterpret_cast<M*>(static_cast<uint16_t*>(base) + off) = w;
    } else if constexpr (BF16 || VEC <= 4) {
        using V = Vec<BF16, VEC>;
        stv<V>(static_cast<typename V::E*>(base) + off, V::pack(v));
    } else {
        using V = Vec<false, 4>;
        float* p = static_cast<float*>(base) + off;
        stv<V>(p, V::T{v[0], v[1], v[2], v[3]});
        stv<V>(p + 4, V::T{v[4], v[5], v[6], v[7]});
    }
}

__device__ __forceinline__ int64_t token_at(const void* ids, int wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(ids)[i] : (int64_t) static_cast<const int32_t*>(ids)[i];
}

// ---- lookup ---------------------------------------------------------------------------
// The output is one run of n * dv vectors (dv per row; the last vector of a
// row that VEC does not divide starts VEC before the row's end and repeats
// some of its neighbour's values).  A workgroup takes 256 * kLook of them
// (2, 4 and 8 measured 8.1, 8.4 and 9.4 us for 50 MB; larger lookups are bound
// by memory with any).
constexpr int kLook = 2;

template <bool BF16, int VEC>
__global__ void __launch_bounds__(256) embed_fwd(EmbedArgs a) {
    using V = Vec<BF16, VEC>;
    using E = typename V::E;
    const uint32_t dv = (uint32_t)((a.D + VEC - 1) / VEC);
    const int64_t first = (int64_t)xcd_logical(blockIdx.x, gridDim.x) * (256 * kLook);
    const int64_t row0 = first / dv;
    const uint32_t rem0 = (uint32_t)(first - row0 * dv);
    typename V::T w[kLook];
    int64_t row[kLook], tok[kLook];
    uint32_t col[kLook];
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
        const uint32_t o = rem0 + j * 256 + threadIdx.x;
        const uint32_t q = o / dv;
        row[j] = row0 + q;
        col[j] = min((o - q * dv) * VEC, (uint32_t)(a.D - VEC));
        tok[j] = row[j] < a.n ? token_at(a.ids, a.wide, row[j]) : -1;
    }
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
        const bool ok = tok[j] >= 0 && tok[j] < a.rows;
        w[j] = typename V::T{};
        if (ok) w[j] = ldv<V>(static_cast<const E*>(a.weight) + tok[j] * a.D + col[j]);
    }
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
        if (row[j] >= a.n) continue;
        float v[VEC];
        V::unpack(w[j], v);
#pragma unroll
        for (int c = 0; c < VEC; ++c) v[c] *= a.scale;
        stv<V>(static_cast<E*>(a.out) + row[j] * a.D + col[j], V::pack(v));
    }
}

// ---- sort -----------------------------------------------------------------------------
// Least significant digit first, a.bits (kDigitBits at most) a pass: count the
// digits of each tile, then place every entry.  Entries of one digit keep their
// order: a wave ranks 64 of them at a time by lane (ballots), adds what it has
// ranked before, and starts after the waves and tiles before it.
constexpr int kDigits = 1 << kDigitBits;

// The sort key of entry i: its token, or `rows` (sorted last, and ignored)
// where the token is out of range or the padding token.
__device__ __forceinline__ uint32_t key_of(const EmbedArgs& a, int64_t i) {
    const int64_t t = token_at(a.ids, a.wide, i);
    return t < 0 || t >= a.rows || t == a.padding ? (uint32_t)a.rows : (uint32_t)t;
}

__device__ __forceinline__ uint32_t pass_key(const EmbedArgs& a, const SortPass& p, int64_t i) {
    return p.first ? key_of(a, i) : p.key_in[i];
}

// lanes of the wave holding the same digit of `bits` bits (of those in `in`)
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint64_t in, int bits) {
    uint32_t lo = (uint32_t)in, hi = (uint32_t)(in >> 32);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        if (b >= bits) break;
        const uint32_t other = ((d >> b) & 1) - 1;  // all ones where the bit is 0
        const uint64_t v = __ballot(other == 0);
        lo &= (uint32_t)v ^ other;
        hi &= (uint32_t)(v >> 32) ^ other;
    }
    return ((uint64_t)hi << 32) | lo;
}

// Entries a thread holds: with 8 a workgroup's chain of rounds is longer (53
// against 46 us for the gradient of 16384 tokens), with 2 the tiles are more
// than what reads their counts likes (648 against 636 us for 131072).
constexpr int kSortRounds = 4;
constexpr int kSubtile = 256 * kSortRounds;  // entries a workgroup places at a time

// hist[tile][digit]
__global__ void __launch_bounds__(256) sort_count(EmbedArgs a, SortPass p) {
    __shared__ uint32_t s_n[kDigits];
    const int64_t i0 = (int64_t)blockIdx.x * a.tile, i1 = min(a.n, i0 + a.tile);
    for (int d = threadIdx.x; d < kDigits; d += 256) s_n[d] = 0;
    __syncthreads();
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSubtile) {
        uint32_t key[kSortRounds];
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) key[r] = pass_key(a, p, min(i + 256 * r, i1 - 1));
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r)
            if (i + 256 * r < i1) atomicAdd(&s_n[(key[r] >> p.shift) & p.mask], 1u);  // whole numbers
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += 256)
        p.hist[(int64_t)blockIdx.x * kDigits + d] = s_n[d];
}

// Among the wave's entries of each round: how many of the digit come before,
// and (bit r of the result) whether this is the last of them; then the same
// over the wave's rounds, with the counts of digits so far in s_n.
template <int ROUNDS, class N>
__device__ __forceinline__ void rank_rounds(const uint32_t (&digit)[ROUNDS], uint32_t in, int rounds,
                                            int bits, int lane, N* s_n, uint32_t (&rank)[ROUNDS]) {
    uint32_t last = 0;
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r >= rounds) break;
        const bool here = (in >> r) & 1;
        const uint64_t m = same_digit(digit[r], __ballot(here), bits);
        rank[r] = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                            __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
        last |= (here && (m >> lane) == 1 ? 1u : 0u) << r;
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r >= rounds) break;
        N* q = s_n + digit[r];
        rank[r] += *q;
        __builtin_amdgcn_wave_barrier();  // read before the digit's last lane counts the round
        if ((last >> r) & 1) *q = (N)(rank[r] + 1);
        __builtin_amdgcn_wave_barrier();
    }
}

__global__ void __launch_bounds__(256) sort_place(EmbedArgs a, SortPass p) {
    __shared__ uint32_t s_n[4][kDigits];  // per wave: counts, then the first place of each digit
    __shared__ uint32_t s_wave[4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.x * a.tile, t1 = min(a.n, t0 + a.tile);
    // a wave takes 64 * kSortRounds neighbouring entries of a subtile
    uint32_t key[kSortRounds], pos[kSortRounds];
    auto load = [&](int64_t sub) {
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            const int64_t i = min(sub + wave * (64 * kSortRounds) + 64 * r + lane, t1 - 1);
            key[r] = pass_key(a, p, i);
            pos[r] = p.first ? (uint32_t)i : p.pos_in[i];
        }
    };
    load(t0);
    // entries of smaller digits everywhere, and of this digit in earlier tiles;
    // a thread takes two neighbouring digits
    static_assert(kDigits == 2 * 256, "two digits a thread");
    uint32_t before[2] = {0, 0}, total[2] = {0, 0};
    {
        const uint2* h = reinterpret_cast<const uint2*>(p.hist) + threadIdx.x;
        constexpr int U = 16;  // tiles whose counts travel together
        for (int k = 0; k < a.tiles; k += U) {
            uint2 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = k + u < a.tiles ? h[(int64_t)(k + u) * (kDigits / 2)] : make_uint2(0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                total[0] += v[u].x;
                total[1] += v[u].y;
                if (k + u < (int)blockIdx.x) before[0] += v[u].x, before[1] += v[u].y;
            }
        }
    }
    const uint32_t sum = total[0] + total[1];
    uint32_t inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t v = __shfl_up(inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 63) s_wave[wave] = inc;
    __syncthreads();
    uint32_t start[2];  // next place of the thread's digits
    start[0] = inc - sum;
    for (int w = 0; w < wave; ++w) start[0] += s_wave[w];
    start[1] = start[0] + total[0] + before[1];
    start[0] += before[0];

    for (int64_t sub = t0; sub < t1; sub += kSubtile) {
        if (sub > t0) load(sub);
        for (int d = threadIdx.x; d < 4 * kDigits; d += 256) (&s_n[0][0])[d] = 0;
        __syncthreads();
        uint32_t digit[kSortRounds], rank[kSortRounds], in = 0;
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            digit[r] = (key[r] >> p.shift) & p.mask;
            in |= (sub + wave * (64 * kSortRounds) + 64 * r + lane < t1 ? 1u : 0u) << r;
        }
        rank_rounds<kSortRounds>(digit, in, kSortRounds, a.bits, lane, s_n[wave], rank);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t v = s_n[w][2 * threadIdx.x + q];
                s_n[w][2 * threadIdx.x + q] = start[q];
                start[q] += v;
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            if ((in >> r) & 1) {
                const uint32_t at = s_n[wave][digit[r]] + rank[r];
                p.key_out[at] = key[r];
                p.pos_out[at] = pos[r];
            }
        }
        __syncthreads();
    }
}

// Up to kSmall entries: one workgroup sorts them whole, in LDS, all passes in
// one launch, in the same manner (the gradient of 5000 rows of 256 bf16 27.4 us
// for 31.3 with four launches, of 8192 equal, of 16384 more: this sort alone
// takes 34 us then).
constexpr int kSmallWaves = 16, kSmallRounds = kSmall / (64 * kSmallWaves);

__global__ void __launch_bounds__(64 * kSmallWaves) sort_small(EmbedArgs a, SortPass p) {
    __shared__ uint32_t s_key[kSmall];
    __shared__ uint16_t s_pos[kSmall];
    __shared__ uint16_t s_n[kSmallWaves][kDigits];  // places stay below kSmall
    __shared__ uint32_t s_wave[kSmallWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = (int)a.n;
    const int rounds = (n + 64 * kSmallWaves - 1) / (64 * kSmallWaves);
    const int i0 = wave * rounds * 64 + lane;  // entry of round r: i0 + 64 r
    uint32_t key[kSmallRounds], digit[kSmallRounds], rank[kSmallRounds], in = 0;
    uint16_t pos[kSmallRounds];
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
        const int i = i0 + 64 * r;
        const bool here = r < rounds && i < n;
        in |= (here ? 1u : 0u) << r;
        key[r] = here ? key_of(a, i) : 0;
        pos[r] = (uint16_t)i;
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        for (int d = tid; d < kSmallWaves * kDigits / 2; d += 64 * kSmallWaves)
            reinterpret_cast<uint32_t*>(&s_n[0][0])[d] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSmallRounds; ++r)
            digit[r] = (key[r] >> (pass * a.bits)) & ((1u << a.bits) - 1);
        rank_rounds<kSmallRounds>(digit, in, rounds, a.bits, lane, s_n[wave], rank);
        __syncthreads();
        // first place of each digit, and of each wave within it
        uint32_t total = 0;
        if (tid < kDigits) {
#pragma unroll
            for (int w = 0; w < kSmallWaves; ++w) total += s_n[w][tid];
        }
        uint32_t inc = total;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t v = __shfl_up(inc, off);
            if (lane >= off) inc += v;
        }
        if (lane == 63) s_wave[wave] = inc;
        __syncthreads();
        if (tid < kDigits) {
            uint32_t at = inc - total;
            for (int w = 0; w < wave; ++w) at += s_wave[w];
#pragma unroll
            for (int w = 0; w < kSmallWaves; ++w) {
                const uint32_t v = s_n[w][tid];
                s_n[w][tid] = (uint16_t)at;
                at += v;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSmallRounds; ++r) {
            if ((in >> r) & 1) {
                const uint32_t at = s_n[wave][digit[r]] + rank[r];
                s_key[at] = key[r];
                s_pos[at] = pos[r];
            }
        }
        __syncthreads();
        if (pass + 1 < a.passes) {
#pragma unroll
            for (int r = 0; r < kSmallRounds; ++r)
                if ((in >> r) & 1) key[r] = s_key[i0 + 64 * r], pos[r] = s_pos[i0 + 64 * r];
        }
    }
    for (int i = tid; i < n; i += 64 * kSmallWaves) {
        p.key_out[i] = s_key[i];
        p.pos_out[i] = s_pos[i];
    }
}

// ---- sums -----------------------------------------------------------------------------
// A group of a.lanes threads (64, 128 or 256: what the columns of one pass
// need) takes a.chunk sorted entries, or kZeroRows rows of the table, by
// a.lanes * VEC columns.  Groups first cover the sorted entries; the rest
// write the zero rows of tokens that do not occur.  (Clearing the gradient in
// the sort's launches, which leave the chip empty, measured 46 against 43 us
// for 16384 rows of 768 bf16: it slows the sort.)  A group for every run of one token instead, with no
// walk over runs, measured twice the time (1350 against 645 us for 131072
// rows of 2048 fp32): its three dependent loads then bring one row.
constexpr int kZeroRows = 16;

// First sorted entry whose key is not below v.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* key, int64_t n, uint32_t v) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (key[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// This thread's piece of work (the same for a wave) and its first column;
// false where the table has no such column.
template <int VEC>
__device__ __forceinline__ bool place(const EmbedArgs& a, int64_t& work, int& col) {
    const int per = 256 / a.lanes;  // groups in a workgroup
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / a.lanes);
    const int64_t l = (int64_t)blockIdx.x * per + group;
    const int32_t cgroups = (a.D + a.lanes * VEC - 1) / (a.lanes * VEC);
    work = l / cgroups;
    col = ((int)(l - work * cgroups) * a.lanes + (int)(threadIdx.x % a.lanes)) * VEC;
    const bool ok = col < a.D;
    col = min(col, a.D - VEC);
    return ok;
}

// Zeros in the rows from v of which none occurs: over their bytes in whole
// vectors, whatever the row's own alignment, with no lanes past the end of a row.
// Row by row instead, stores cross lines: 126108 rows of 1530 fp32 with 300 entries
// 208 us for 163 (of 1536 157 for 151), 40296 of 2115 bf16 with 5206 63 for 50, and
// the same where most rows occur.
template <int VEC, bool GBF16>
__device__ __forceinline__ void clear_rows(const EmbedArgs& a, int64_t v, int rows) {
    using G = typename std::conditional<GBF16, uint16_t, float>::type;
    constexpr int N = 16 / sizeof(G);
    const int lanes = a.lanes, per = 256 / lanes;
    const int cgroups = (a.D + lanes * VEC - 1) / (lanes * VEC);
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / lanes);
    const int piece = (int)(((int64_t)blockIdx.x * per + group) % cgroups);
    const int64_t at = piece * (int64_t)lanes + threadIdx.x % lanes;
    const int64_t step = (int64_t)cgroups * lanes;
    const int64_t e0 = v * a.D, e1 = e0 + (int64_t)rows * a.D;
    const int64_t v0 = (e0 + N - 1) / N, v1 = e1 / N;  // its whole vectors
    G* g = static_cast<G*>(a.dweight);
    for (int64_t i = v0 + at; i < v1; i += step) reinterpret_cast<uint4*>(g)[i] = uint4{0, 0, 0, 0};
    const int64_t head = min(v0 * N, e1), tail = max(v1 * N, head);
    if (e0 + at < head) g[e0 + at] = 0;
    if (tail + at < e1) g[tail + at] = 0;
}

template <bool BF16, int VEC, bool GBF16>
__global__ void __launch_bounds__(256) embed_sum(EmbedArgs a, const uint32_t* key,
                                                 const uint32_t* pos) {
    using V = Vec<BF16, VEC>;
    using E = typename V::E;
    int64_t work;
    int col;
    const bool live = place<VEC>(a, work, col);
    if (work >= a.chunks + a.zeros) return;
    if (work >= a.chunks) {
        const int64_t v0 = (work - a.chunks) * kZeroRows;
        // lane k of the wave finds out whether token v0 + k occurs
        const int64_t v = v0 + (threadIdx.x & (kZeroRows - 1));
        bool has = true;  // nothing to write past the table
        if (v < a.rows) {
            const int64_t at = lower_bound(key, a.n, (uint32_t)v);
            has = at < a.n && key[at] == (uint32_t)v;
        }
        const uint64_t m = __ballot(has);
        uint32_t none = ~(uint32_t)m & ((1u << kZeroRows) - 1);
        while (none) {
            const int k = __ffs(none) - 1, n = __ffs(~(none >> k)) - 1;
            clear_rows<VEC, GBF16>(a, v0 + k, n);
            none &= ~(((1u << n) - 1) << k);
        }
        return;
    }
    const int64_t e0 = work * a.chunk, e1 = min(a.n, e0 + a.chunk);
    // a run that starts before the chunk, or goes on after it, leaves a part
    const uint32_t prev = e0 > 0 ? key[e0 - 1] : 0xffffffffu;
    const uint32_t next = e1 < a.n ? key[e1] : 0xffffffffu;
    const int lane = threadIdx.x & 63;
    float acc[VEC] = {};
    uint32_t cur = key[e0];
    bool head = cur == prev;  // the current run began in an earlier chunk
    auto flush = [&](bool goes_on) {
        if (cur >= (uint32_t)a.rows || !live) return;  // ignored entries, columns past the row
        if (head || goes_on) {
            float* q = a.part + (2 * work + (head ? 0 : 1)) * (int64_t)a.D + col;
#pragma unroll
            for (int c = 0; c < VEC; ++c) q[c] = acc[c];
        } else {
            float v[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[c] = acc[c] * a.scale;
            store_grad<VEC, GBF16>(a.dweight, (int64_t)cur * a.D + col, v);
        }
    };
    const E* dy = static_cast<const E*>(a.dy) + col;
    constexpr int U = 8;  // rows on the way at a time
    for (int64_t b = e0; b < e1; b += 64) {
        // a lane an entry, so that all positions arrive together; then one
        // entry after another, the same for the whole wave
        const int64_t at = min(b + lane, e1 - 1);
        const uint32_t kl = key[at], pl = pos[at];
        const int m = (int)min(e1 - b, (int64_t)64);
        for (int e = 0; e < m; e += U) {
            typename V::T w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t row = __builtin_amdgcn_readlane(pl, min(e + u, 63));
                w[u] = ldv<V>(dy + (int64_t)row * a.D);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (e + u >= m) break;
                const uint32_t k = __builtin_amdgcn_readlane(kl, e + u);
                if (k != cur) {
                    flush(false);
                    cur = k;
                    head = false;
#pragma unroll
                    for (int c = 0; c < VEC; ++c) acc[c] = 0.f;
                }
                float v[VEC];
                V::unpack(w[u], v);
#pragma unroll
                for (int c = 0; c < VEC; ++c) acc[c] += v[c];
            }
        }
    }
    flush(cur == next);
}

// Joins the pieces of runs that cross chunks: the group of the chunk where a
// run starts adds its tail part and the head parts of the chunks after it, in
// order, with kJoin of them on the way at a time.
constexpr int kJoin = 16;

template <int VEC, bool GBF16>
__global__ void __launch_bounds__(256) embed_join(EmbedArgs a, const uint32_t* key) {
    int64_t work;
    int col;
    const bool live = place<VEC>(a, work, col);
    if (work >= a.chunks - 1) return;  // the last chunk starts nothing that goes on
    const int64_t e0 = work * a.chunk, e1 = e0 + a.chunk;
    const uint32_t run = key[e1 - 1];
    if (run >= (uint32_t)a.rows || key[e1] != run) return;  // nothing goes on
    if (e0 > 0 && key[e0 - 1] == run) return;               // it started before this chunk
    // the chunk of its last entry: the chunks after this one that begin with it
    int64_t last = work;
    for (;;) {
        const int64_t k = last + 1 + (threadIdx.x & 63);
        const uint64_t other = ~__ballot(k < a.chunks && key[k * a.chunk] == run);
        if (other) {
            last += __ffsll((unsigned long long)other) - 1;
            break;
        }
        last += 64;
    }
    if (!live) return;
    const int64_t D = a.D;
    float acc[VEC];
    const float* q = a.part + (2 * work + 1) * D + col;
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] = q[c];
    int64_t k = work + 1;
    for (; k + kJoin <= last + 1; k += kJoin) {
        float v[kJoin][VEC];
#pragma unroll
        for (int u = 0; u < kJoin; ++u)
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[u][c] = a.part[2 * (k + u) * D + col + c];
#pragma unroll
        for (int u = 0; u < kJoin; ++u)
#pragma unroll
            for (int c = 0; c < VEC; ++c) acc[c] += v[u][c];
    }
    for (; k <= last; ++k) {
        q = a.part + 2 * k * D + col;
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[c] += q[c];
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] *= a.scale;
    store_grad<VEC, GBF16>(a.dweight, (int64_t)run * D + col, acc);
}

// Up to kFew entries: no sort, one launch for three.  Groups first cover the
// entries: the group of a token's first entry sums them all in order.  The other
// workgroups take the gradient's bytes in order, a vector a lane, and write zeros
// where no entry's row lies: memory takes stores best in the order of workgroups
// (775 MB 115 us with 4 KB a workgroup, 128 with 8 or 16, 143 with 96).  19 entries in
// 126108 rows of 1530 fp32 110 us for 150 with 16 rows a group, 64 of 768 bf16 in
// 50280 14.8 for 16.3.  K entries a lane, that each wave looks through: with 4 up to 128
// entries take 125 and 18 there; 200 entries 130 and 19, sorted 163 and 25, with 8
// 215 and 27.
template <bool BF16, int VEC, bool GBF16, int K>
__global__ void __launch_bounds__(256) embed_few(EmbedArgs a) {
    using V = Vec<BF16, VEC>;
    using E = typename V::E;
    const int lane = threadIdx.x & 63, n = (int)a.n;
    int64_t t[K];  // a lane's entries: their rows, or -1
#pragma unroll
    for (int k = 0; k < K; ++k) {
        t[k] = k * 64 + lane < n ? token_at(a.ids, a.wide, k * 64 + lane) : -1;
        if (t[k] < 0 || t[k] >= a.rows || t[k] == a.padding) t[k] = -1;
    }
    if (blockIdx.x >= a.sums) {
        using G = typename std::conditional<GBF16, uint16_t, float>::type;
        constexpr int N = 16 / sizeof(G);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int64_t all = a.rows * a.D;
        const int64_t e0 = (((int64_t)blockIdx.x - a.sums) * 4 + wave) * 64 * N;
        const int64_t e = e0 + lane * N;
        uint32_t take = 0;  // elements of this lane's vector that lie in an entry's row
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t s0 = t[k] * a.D;
            const bool in = t[k] >= 0 && s0 < e0 + 64 * N && s0 + a.D > e0;
            for (uint64_t m = __ballot(in); m; m &= m - 1) {
                const int64_t r0 = __shfl(s0, __ffsll((unsigned long long)m) - 1);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (e + j >= r0 && e + j < r0 + a.D) take |= 1u << j;
            }
        }
        G* g = static_cast<G*>(a.dweight) + e;
        if (!take && e + N <= all) {
            *reinterpret_cast<uint4*>(g) = uint4{0, 0, 0, 0};
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (!((take >> j) & 1) && e + j < all) g[j] = 0;
        }
        return;
    }
    int64_t work;
    int col;
    const bool live = place<VEC>(a, work, col);
    if (work >= a.chunks) return;  // chunks are entries here
    int64_t row = -1;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (work >> 6 == k) row = __shfl(t[k], (int)(work & 63));
    if (row < 0) return;
    uint64_t m[K];
    bool first = true;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        m[k] = __ballot(t[k] == row);
        const int64_t before = work - k * 64;
        if (before >= 64 ? m[k] != 0 : before > 0 && (m[k] & ((1ull << before) - 1))) first = false;
    }
    if (!first) return;
    const E* dy = static_cast<const E*>(a.dy) + col;
    constexpr int U = 8;  // rows on the way at a time
    float acc[VEC] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        while (m[k]) {
            typename V::T w[U];
            int got = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!m[k]) break;
                const int at = k * 64 + __ffsll((unsigned long long)m[k]) - 1;
                m[k] &= m[k] - 1;
                w[u] = ldv<V>(dy + (int64_t)at * a.D);
                ++got;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u >= got) break;
                float v[VEC];
                V::unpack(w[u], v);
#pragma unroll
                for (int c = 0; c < VEC; ++c) acc[c] += v[c];
            }
        }
    }
    if (!live) return;
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] *= a.scale;
    store_grad<VEC, GBF16>(a.dweight, row * a.D + col, acc);
}

template <bool BF16, int VEC>
hipError_t sum_variant(const EmbedArgs& a, bool gbf16, const uint32_t* key, const uint32_t* pos,
                       hipStream_t s) {
    const int64_t cgroups = (a.D + a.lanes * VEC - 1) / (a.lanes * VEC), per = 256 / a.lanes;
    const dim3 grid((unsigned)embed_sum_workgroups(a, BF16, gbf16)), blk(256);
    if (a.few) {
        ProfScope ps(s, kPhaseMain);
        auto go = [&](auto k) {
            constexpr int K = decltype(k)::value;
            if (gbf16) hipLaunchKernelGGL((embed_few<BF16, VEC, true, K>), grid, blk, 0, s, a);
            else hipLaunchKernelGGL((embed_few<BF16, VEC, false, K>), grid, blk, 0, s, a);
        };
        constexpr int most = kFew / 64;
        if (a.n <= kFew / 2) go(std::integral_constant<int, most / 2>{});
        else go(std::integral_constant<int, most>{});
        return hipGetLastError();
    }
    {
        ProfScope ps(s, kPhaseMain);
        if (gbf16) hipLaunchKernelGGL((embed_sum<BF16, VEC, true>), grid, blk, 0, s, a, key, pos);
        else hipLaunchKernelGGL((embed_sum<BF16, VEC, false>), grid, blk, 0, s, a, key, pos);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.chunks < 2) return e;
    ProfScope ps(s, kPhaseReduce);
    const dim3 jgrid((unsigned)(((a.chunks - 1) * cgroups + per - 1) / per));
    if (gbf16) hipLaunchKernelGGL((embed_join<VEC, true>), jgrid, blk, 0, s, a, key);
    else hipLaunchKernelGGL((embed_join<VEC, false>), jgrid, blk, 0, s, a, key);
    return hipGetLastError();
}

}  // namespace

int embed_vec(int D, bool bf16) {
    const int v = bf16 ? 8 : 4;
    return D >= v ? v : 1;
}

int64_t embed_sum_workgroups(const EmbedArgs& a, bool bf16, bool gbf16) {
    if (!a.few) {
        const int64_t vec = embed_vec(a.D, bf16), cols = a.lanes * vec, per = 256 / a.lanes;
        return ((a.chunks + a.zeros) * ((a.D + cols - 1) / cols) + per - 1) / per;
    }
    const int64_t span = 256 * (gbf16 ? 8 : 4);  // elements
    return a.sums + (a.rows * a.D + span - 1) / span;
}

int64_t embed_fwd_workgroups(const EmbedArgs& a, bool bf16) {
    const int64_t v = embed_vec(a.D, bf16);
    const double vecs = (double)a.n * (double)((a.D + v - 1) / v);
    return vecs > 0x1p50 ? INT64_MAX : ((int64_t)vecs + 256 * kLook - 1) / (256 * kLook);
}

hipError_t launch_embed_fwd(const EmbedArgs& a, bool bf16, hipStream_t s) {
    ProfScope ps(s, kPhaseMain);
    const dim3 grid((unsigned)embed_fwd_workgroups(a, bf16)), blk(256);
    if (embed_vec(a.D, bf16) > 1) {
        if (bf16) hipLaunchKernelGGL((embed_fwd<true, 8>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((embed_fwd<false, 4>), grid, blk, 0, s, a);
    } else {
        if (bf16) hipLaunchKernelGGL((embed_fwd<true, 1>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((embed_fwd<false, 1>), grid, blk, 0, s, a);
    }
    return hipGetLastError();
}

void embed_plan(EmbedArgs& a, bool bf16) {
    // at most kMaxTiles tiles, so that a workgroup of sort_place reads the
    // whole count matrix from L2 in little time
    const int64_t quantum = kSubtile;
    int64_t tile = (a.n + kMaxTiles - 1) / kMaxTiles;
    tile = (tile + quantum - 1) / quantum * quantum;
    a.tile = tile < quantum ? quantum : tile;
    a.tiles = (int)((a.n + a.tile - 1) / a.tile);
    int bits = 1;  // keys run from 0 to rows
    while (bits < 32 && ((uint64_t)a.rows >> bits) != 0) ++bits;
    a.passes = (bits + kDigitBits - 1) / kDigitBits;
    a.bits = (bits + a.passes - 1) / a.passes;
    const int vec = embed_vec(a.D, bf16);
    const int64_t vecs = (a.D + vec - 1) / vec;
    a.lanes = vecs <= 64 ? 64 : vecs <= 128 ? 128 : 256;
    // chunks: enough groups to fill the chip, long enough that a frequent
    // token's run has few pieces to join
    const int64_t cgroups = (vecs + a.lanes - 1) / a.lanes;
    const int64_t chunk = a.n * cgroups * a.lanes / (2048 * 256);
    a.chunk = chunk < 32 ? 32 : chunk > 256 ? 256 : chunk;
    a.chunks = (a.n + a.chunk - 1) / a.chunk;
    // a table whose vectors are too many for one launch is sorted for
    a.few = a.n <= kFew && (double)a.rows * a.D <= 0x1p33;
    if (a.few) a.chunks = a.n;
    a.small = a.n <= kSmall;
    const int64_t per = 256 / a.lanes;
    a.sums = (a.chunks * cgroups + per - 1) / per;
    a.zeros = (a.rows + kZeroRows - 1) / kZeroRows;
}

// [hist][key x2][pos x2][parts], 256-byte aligned regions
EmbedWs embed_ws(const EmbedArgs& a) {
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    EmbedWs w{};
    if (a.few) return w;
    w.hist = 0;
    size_t off = up((size_t)a.tiles * kDigits * 4);
    for (int k = 0; k < 2; ++k) {
        w.key[k] = off;
        off += up((size_t)a.n * 4);
        w.pos[k] = off;
        off += up((size_t)a.n * 4);
    }
    w.part = off;
    off += a.chunks > 1 ? up((size_t)a.chunks * 2 * (size_t)a.D * 4) : 0;
    w.total = off;
    return w;
}

hipError_t launch_embed_bwd(EmbedArgs a, bool bf16, bool gbf16, void* workspace, hipStream_t s) {
    char* ws = static_cast<char*>(workspace);
    const EmbedWs w = embed_ws(a);
    a.part = reinterpret_cast<float*>(ws + w.part);
    int out = 0;
    SortPass p{};
    p.hist = reinterpret_cast<uint32_t*>(ws + w.hist);
    for (int k = 0; !a.few && k < (a.small ? 1 : a.passes); ++k) {
        p.first = k == 0;
        p.shift = k * a.bits;
        p.mask = (1u << a.bits) - 1;
        out = k & 1;
        p.key_in = reinterpret_cast<uint32_t*>(ws + w.key[out ^ 1]);
        p.pos_in = reinterpret_cast<uint32_t*>(ws + w.pos[out ^ 1]);
        p.key_out = reinterpret_cast<uint32_t*>(ws + w.key[out]);
        p.pos_out = reinterpret_cast<uint32_t*>(ws + w.pos[out]);
        ProfScope ps(s, kPhasePrep);
        if (a.small) {
            hipLaunchKernelGGL(sort_small, dim3(1), dim3(64 * kSmallWaves), 0, s, a, p);
        } else {
            hipLaunchKernelGGL(sort_count, dim3(a.tiles), dim3(256), 0, s, a, p);
            hipLaunchKernelGGL(sort_place, dim3(a.tiles), dim3(256), 0, s, a, p);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const uint32_t* key = reinterpret_cast<uint32_t*>(ws + w.key[out]);
    const uint32_t* pos = reinterpret_cast<uint32_t*>(ws + w.pos[out]);
    if (embed_vec(a.D, bf16) > 1)
        return bf16 ? sum_variant<true, 8>(a, gbf16, key, pos, s)
                    : sum_variant<false, 4>(a, gbf16, key, pos, s);
    return bf16 ? sum_variant<true, 1>(a, gbf16, key, pos, s)
                : sum_variant<false, 1>(a, gbf16, key, pos, s);
}

}  // namespace msscan
