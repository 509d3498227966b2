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
#include <hip/hip_runtime.h>
#include <stdint.h>

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
// some of its neighbour's values).  A workgroup takes 256 * kLook of them.
constexpr int kLook = 4;

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
// Least significant digit first, kDigitBits at most a pass.  A workgroup
// takes a.tile consecutive entries, each of its waves a quarter of them in
// order; entries of one digit keep their order because a wave ranks 64 of
// them at a time by lane (ballots), adds what it has placed before, and starts
// after the waves and workgroups before it.
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

// lanes of the wave holding the same digit (of those in `in`)
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint64_t in) {
    uint64_t m = in;
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        const uint64_t v = __ballot((d >> b) & 1);
        m &= ((d >> b) & 1) ? v : ~v;
    }
    return m;
}

// hist[tile][digit]
__global__ void __launch_bounds__(256) sort_count(EmbedArgs a, SortPass p) {
    __shared__ uint32_t s_n[kDigits];
    for (int d = threadIdx.x; d < kDigits; d += 256) s_n[d] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * a.tile, i1 = min(a.n, i0 + a.tile);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += 256)
        atomicAdd(&s_n[(pass_key(a, p, i) >> p.shift) & (kDigits - 1)], 1u);  // whole numbers
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += 256)
        p.hist[(int64_t)blockIdx.x * kDigits + d] = s_n[d];
}

__global__ void __launch_bounds__(256) sort_place(EmbedArgs a, SortPass p) {
    __shared__ uint32_t s_n[4][kDigits];  // per wave: counts, then the next place of each digit
    __shared__ uint32_t s_wave[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int d = threadIdx.x; d < 4 * kDigits; d += 256) (&s_n[0][0])[d] = 0;
    __syncthreads();
    const int64_t part = a.tile / 4;
    const int64_t i0 = min(a.n, (int64_t)blockIdx.x * a.tile + wave * part);
    const int64_t i1 = min(a.n, i0 + part);
    for (int64_t i = i0 + lane; i < i1; i += 64)
        atomicAdd(&s_n[wave][(pass_key(a, p, i) >> p.shift) & (kDigits - 1)], 1u);
    // entries of smaller digits everywhere, and of this digit in earlier tiles
    constexpr int PER = kDigits / 256;
    uint32_t before[PER], total[PER], sum = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        before[q] = total[q] = 0;
        const uint32_t* h = p.hist + threadIdx.x * PER + q;
        for (int t = 0; t < a.tiles; ++t) {
            const uint32_t v = h[(int64_t)t * kDigits];
            total[q] += v;
            if (t < (int)blockIdx.x) before[q] += v;
        }
        sum += total[q];
    }
    uint32_t inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t v = __shfl_up(inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 63) s_wave[wave] = inc;
    __syncthreads();
    uint32_t at = inc - sum;
    for (int w = 0; w < wave; ++w) at += s_wave[w];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int d = threadIdx.x * PER + q;
        uint32_t place = at + before[q];
        for (int w = 0; w < 4; ++w) {
            const uint32_t v = s_n[w][d];
            s_n[w][d] = place;
            place += v;
        }
        at += total[q];
    }
    __syncthreads();
    for (int64_t i = i0; i < i1; i += 64) {
        const bool in = i + lane < i1;
        const uint32_t key = in ? pass_key(a, p, i + lane) : 0;
        const uint32_t d = (key >> p.shift) & (kDigits - 1);
        const uint64_t m = same_digit(d, __ballot(in));
        uint32_t place = 0;
        if (in) place = s_n[wave][d] + __popcll(m & ((1ull << lane) - 1));
        // all lanes have read the place before its last holder moves it on
        __builtin_amdgcn_wave_barrier();
        if (in && (m >> lane) == 1) s_n[wave][d] = place + 1;
        __builtin_amdgcn_wave_barrier();
        if (in) {
            p.key_out[place] = key;
            p.pos_out[place] = p.first ? (uint32_t)(i + lane) : p.pos_in[i + lane];
        }
    }
}

// ---- sums -----------------------------------------------------------------------------
// Workgroups first cover the sorted entries, a.chunk of them by 256 * VEC
// columns each; the rest write the zero rows of tokens that do not occur,
// kZeroRows rows by 256 * VEC columns each.
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

template <bool BF16, int VEC, bool GBF16>
__global__ void __launch_bounds__(256) embed_sum(EmbedArgs a, const uint32_t* key,
                                                 const uint32_t* pos) {
    using V = Vec<BF16, VEC>;
    using E = typename V::E;
    const int32_t cgroups = (a.D + 256 * VEC - 1) / (256 * VEC);
    const int64_t l = blockIdx.x;
    const int64_t work = l / cgroups;
    const int cg = (int)(l - work * cgroups);
    int col = (cg * 256 + (int)threadIdx.x) * VEC;
    const bool live = col < a.D;
    col = min(col, a.D - VEC);
    if (work >= a.chunks) {
        __shared__ int s_has[kZeroRows];
        const int64_t v0 = (work - a.chunks) * kZeroRows;
        if (threadIdx.x < kZeroRows) {
            const int64_t v = v0 + threadIdx.x;
            int has = 1;  // nothing to write past the table
            if (v < a.rows) {
                const int64_t at = lower_bound(key, a.n, (uint32_t)v);
                has = at < a.n && key[at] == (uint32_t)v;
            }
            s_has[threadIdx.x] = has;
        }
        __syncthreads();
        if (!live) return;
        const float zero[VEC] = {};
        for (int k = 0; k < kZeroRows; ++k)
            if (!s_has[k]) store_grad<VEC, GBF16>(a.dweight, (v0 + k) * a.D + col, zero);
        return;
    }
    if (!live) return;
    const int64_t e0 = work * a.chunk, e1 = min(a.n, e0 + a.chunk);
    // a run that starts before the chunk, or goes on after it, leaves a part
    const uint32_t prev = e0 > 0 ? key[e0 - 1] : 0xffffffffu;
    const uint32_t next = e1 < a.n ? key[e1] : 0xffffffffu;
    float acc[VEC] = {};
    uint32_t cur = key[e0];
    bool head = cur == prev;  // the current run began in an earlier chunk
    auto flush = [&](bool goes_on) {
        if (cur >= (uint32_t)a.rows) return;  // ignored entries
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
    constexpr int U = 8;
    for (int64_t e = e0; e < e1; e += U) {
        typename V::T w[U];
        uint32_t kk[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = min(e + u, e1 - 1);
            kk[u] = key[at];
            w[u] = ldv<V>(dy + (int64_t)pos[at] * a.D);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (e + u >= e1) break;
            if (kk[u] != cur) {
                flush(false);
                cur = kk[u];
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
    flush(cur == next);
}

// Joins the pieces of runs that cross chunks: the workgroup of the chunk where
// a run starts adds its tail part and the head parts of the chunks after it,
// in order.
template <int VEC, bool GBF16>
__global__ void __launch_bounds__(256) embed_join(EmbedArgs a, const uint32_t* key) {
    const int32_t cgroups = (a.D + 256 * VEC - 1) / (256 * VEC);
    const int64_t work = blockIdx.x / cgroups;
    const int cg = (int)(blockIdx.x - work * cgroups);
    int col = (cg * 256 + (int)threadIdx.x) * VEC;
    if (col >= a.D) return;
    col = min(col, a.D - VEC);
    const int64_t e0 = work * a.chunk, e1 = e0 + a.chunk;
    if (e1 >= a.n) return;  // the last chunk starts nothing that goes on
    const uint32_t run = key[e1 - 1];
    if (run >= (uint32_t)a.rows || key[e1] != run) return;  // nothing goes on
    if (e0 > 0 && key[e0 - 1] == run) return;               // it started before this chunk
    const int64_t end = lower_bound(key, a.n, run + 1);     // one past the run
    const int64_t last = (end - 1) / a.chunk;               // the chunk of its last entry
    float acc[VEC];
    const float* q = a.part + (2 * work + 1) * (int64_t)a.D + col;
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] = q[c];
    for (int64_t k = work + 1; k <= last; ++k) {
        q = a.part + 2 * k * (int64_t)a.D + col;
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[c] += q[c];
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] *= a.scale;
    store_grad<VEC, GBF16>(a.dweight, (int64_t)run * a.D + col, acc);
}

template <bool BF16, int VEC>
hipError_t sum_variant(const EmbedArgs& a, bool gbf16, const uint32_t* key, const uint32_t* pos,
                       hipStream_t s) {
    const int64_t cgroups = (a.D + 256 * VEC - 1) / (256 * VEC);
    const int64_t zero = (a.rows + kZeroRows - 1) / kZeroRows;
    const dim3 grid((unsigned)((a.chunks + zero) * cgroups)), blk(256);
    {
        ProfScope ps(s, kPhaseMain);
        if (gbf16) hipLaunchKernelGGL((embed_sum<BF16, VEC, true>), grid, blk, 0, s, a, key, pos);
        else hipLaunchKernelGGL((embed_sum<BF16, VEC, false>), grid, blk, 0, s, a, key, pos);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.chunks < 2) return e;
    ProfScope ps(s, kPhaseReduce);
    const dim3 jgrid((unsigned)((a.chunks - 1) * cgroups));
    if (gbf16) hipLaunchKernelGGL((embed_join<VEC, true>), jgrid, blk, 0, s, a, key);
    else hipLaunchKernelGGL((embed_join<VEC, false>), jgrid, blk, 0, s, a, key);
    return hipGetLastError();
}

}  // namespace

int embed_vec(int D, bool bf16) {
    const int v = bf16 ? 8 : 4;
    return D >= v ? v : 1;
}

int64_t embed_sum_workgroups(const EmbedArgs& a, bool bf16) {
    const int64_t per = 256 * (int64_t)embed_vec(a.D, bf16);
    return (a.chunks + (a.rows + kZeroRows - 1) / kZeroRows) * ((a.D + per - 1) / per);
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

void embed_plan(EmbedArgs& a) {
    // at most kMaxTiles tiles, so that a workgroup of sort_place reads the
    // whole count matrix from L2 in little time
    const int64_t quantum = 2048;
    int64_t tile = (a.n + kMaxTiles - 1) / kMaxTiles;
    tile = (tile + quantum - 1) / quantum * quantum;
    a.tile = tile < quantum ? quantum : tile;
    a.tiles = (int)((a.n + a.tile - 1) / a.tile);
    int bits = 1;  // keys run from 0 to rows
    while (bits < 32 && ((uint64_t)a.rows >> bits) != 0) ++bits;
    a.passes = (bits + kDigitBits - 1) / kDigitBits;
    a.chunk = 32;
    a.chunks = (a.n + a.chunk - 1) / a.chunk;
}

// [hist][key x2][pos x2][parts], 256-byte aligned regions
EmbedWs embed_ws(const EmbedArgs& a) {
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    EmbedWs w{};
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
    if (a.n > 0) {
        for (int k = 0; k < a.passes; ++k) {
            SortPass p{};
            p.first = k == 0;
            p.shift = k * kDigitBits;
            p.hist = reinterpret_cast<uint32_t*>(ws + w.hist);
            out = k & 1;
            p.key_in = reinterpret_cast<uint32_t*>(ws + w.key[out ^ 1]);
            p.pos_in = reinterpret_cast<uint32_t*>(ws + w.pos[out ^ 1]);
            p.key_out = reinterpret_cast<uint32_t*>(ws + w.key[out]);
            p.pos_out = reinterpret_cast<uint32_t*>(ws + w.pos[out]);
            ProfScope ps(s, kPhasePrep);
            hipLaunchKernelGGL(sort_count, dim3(a.tiles), dim3(256), 0, s, a, p);
            hipLaunchKernelGGL(sort_place, dim3(a.tiles), dim3(256), 0, s, a, p);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
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
