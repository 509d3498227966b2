// group_norm.hip -- norm of each row's channels in groups (the heads of a linear
// attention), with scale, shift and a silu gate, and its gradient:
//
//   u = x, or x silu(z) (gate first)      c = u - mean(u), or u
//   hat = c / sqrt(mean(c^2) + eps)       y = (hat w + b) [silu(z)]
//
// Bytes are all that counts: every input is read once, in vectors of 16 bytes,
// and kept in registers from the sums to the output.  A group is shared by the
// fewest lanes (a power of two) that hold it in one vector each, up to a wave
// with 2 vectors, and by a workgroup beyond that; the groups of a wave lie side
// by side in a row.  A wave keeps its channels and goes down the rows: the
// weights are read once, and the gradients of weights add up in registers.
// They are joined over waves in LDS and over workgroups by a second launch, in
// fixed orders.
//
// 16384 rows of 1536 bf16 with a gate: forward 31 us (4.9 TB/s), backward of one
// group 51 us (4.9 TB/s) and 5 for the join.
#include <type_traits>

#include "device_common.h"
#include "lm_internal.h"
#include "msscan_internal.h"

namespace msscan {
namespace norm {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef u4 u4_align2 __attribute__((aligned(2)));
typedef u4 u4_align4 __attribute__((aligned(4)));

// A barrier for what waves share in LDS, which does not wait for loads and stores
// of global memory under way.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <bool BF16>
constexpr int vec() { return BF16 ? 8 : 4; }

// A vector of a group's values from place i on of n.  ask() has no branch, which
// would wait for its loads: it takes a whole vector that is there, and take()
// moves a group's last values down to where they belong (WHOLE: n is a multiple of
// the vector, and none has to) and clears what lies behind the end.
template <bool BF16, bool WHOLE>
struct Vec {
    static constexpr int W = vec<BF16>();
    typedef typename std::conditional<BF16, uint16_t, float>::type E;
    typedef typename std::conditional<BF16, u4_align2, u4_align4>::type U;
    union {
        float v[W];
        uint32_t raw[4];
    };

    __device__ __forceinline__ void ask(const void* row, int64_t at, int i, int n) {
        const E* p = static_cast<const E*>(row) + at;
        if (WHOLE || n >= W) {
            const u4 x = *reinterpret_cast<const U*>(p + min(i, n - W));
#pragma unroll
            for (int e = 0; e < 4; ++e) raw[e] = x[e];
        } else {  // groups smaller than a vector
#pragma unroll
            for (int e = 0; e < 4; ++e) raw[e] = 0;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const uint32_t x = e < n ? bits(p[min(e, n - 1)]) : 0;
                if constexpr (BF16) raw[e / 2] |= x << (e % 2 * 16);
                else raw[e] = x;
            }
        }
    }
    static __device__ __forceinline__ uint32_t bits(uint16_t x) { return x; }
    static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
    __device__ __forceinline__ void take(int i, int n) {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = raw[e];
        if (!WHOLE && n >= W) {
            const int s = min(max(i + W - n, 0), W);  // values to move down by
            if constexpr (BF16) {
                const bool one = s & 1, two = s & 2, four = s & 4;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = one ? x[e] >> 16 | (e < 3 ? x[e + 1] << 16 : 0) : x[e];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = two ? (e < 3 ? x[e + 1] : 0) : x[e];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = four ? (e < 2 ? x[e + 2] : 0) : x[e];
            } else {
                const bool one = s & 1, two = s & 2;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = one ? (e < 3 ? x[e + 1] : 0) : x[e];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = two ? (e < 2 ? x[e + 2] : 0) : x[e];
            }
        }
        const bool in = i < n;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = in ? x[e] : 0;
#pragma unroll
        for (int e = 0; e < W; ++e)
            if constexpr (BF16)
                v[e] = __uint_as_float(e & 1 ? x[e / 2] & 0xffff0000u : x[e / 2] << 16);
            else
                v[e] = __uint_as_float(x[e]);
    }
    __device__ __forceinline__ void store(void* row, int64_t at, int i, int n) const {
        E* p = static_cast<E*>(row) + at + i;
        if (WHOLE ? i < n : i + W <= n) {
            u4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if constexpr (BF16)
                    x[e] = (uint32_t)f32_to_bf16_rne(v[2 * e]) |
                           (uint32_t)f32_to_bf16_rne(v[2 * e + 1]) << 16;
                else
                    x[e] = __float_as_uint(v[e]);
            *reinterpret_cast<U*>(p) = x;
        } else if (!WHOLE) {
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (i + e < n) st<BF16>(p, e, v[e]);
        }
    }
    // a row of fp32 values that are the same for every row (or `other`)
    __device__ __forceinline__ void weights(const float* row, int64_t at, int i, int n,
                                            float other) {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = row ? row[at + min(i + e, n - 1)] : other;
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = i + e < n ? v[e] : 0.f;
    }
};

enum { kNone = 0, kAfter = 1, kFirst = 2 };  // the gate

// Where a lane works: its first vector's place in its group, and its group.
template <bool WIDE>
struct Lane {
    int first, group, lanes;
    float* scratch;  // two buffers of kWaves
    int turn;        // of the next sum
    __device__ __forceinline__ Lane(const NormArgs& a, float* sums) : scratch(sums), turn(0) {
        lanes = a.lanes;
        if (WIDE) {
            first = threadIdx.x;
            group = blockIdx.x % a.columns;
        } else {
            const int l = threadIdx.x & 63;
            first = l & (lanes - 1);
            group = (blockIdx.x % a.columns) * (64 / lanes) + l / lanes;
        }
    }
    // Over the lanes of a group.  Each sum takes the buffer that the last one did
    // not, whoever calls it: a wave that writes into one has passed the barrier of
    // the sum between, and so have all waves read the sum before that.
    __device__ __forceinline__ float sum(float x) {
        for (int d = 1; d < (WIDE ? 64 : lanes); d *= 2) x += __shfl_xor(x, d);
        if (WIDE) {
            float* part = scratch + turn;
            turn ^= kWaves;
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
            lds_barrier();
            x = (part[0] + part[1]) + (part[2] + part[3]);
        }
        return x;
    }
};

__device__ __forceinline__ float sigmoid(float z) {
    return hw_rcp(1.f + hw_exp2(-z * kLog2e));
}

// The normalised values of a group in place of u, and the factor they took.
template <bool BF16, int NV, bool WIDE, bool WHOLE>
__device__ __forceinline__ float normalise(const NormArgs& a, Lane<WIDE>& at,
                                           Vec<BF16, WHOLE> (&u)[NV]) {
    constexpr int W = vec<BF16>();
    const float inv = 1.f / (float)a.size;
    if (a.center) {
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < NV; ++m)
#pragma unroll
            for (int e = 0; e < W; ++e) s += u[m].v[e];
        const float mean = at.sum(s) * inv;
#pragma unroll
        for (int m = 0; m < NV; ++m)
#pragma unroll
            for (int e = 0; e < W; ++e)
                u[m].v[e] = (at.first + m * at.lanes) * W + e < a.size ? u[m].v[e] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < NV; ++m)
#pragma unroll
        for (int e = 0; e < W; ++e) s = fmaf(u[m].v[e], u[m].v[e], s);
    const float factor = 1.f / sqrtf(fmaf(at.sum(s), inv, a.eps));
#pragma unroll
    for (int m = 0; m < NV; ++m)
#pragma unroll
        for (int e = 0; e < W; ++e) u[m].v[e] *= factor;
    return factor;
}

template <bool BF16, int NV, bool WIDE, bool WHOLE, int GATE, bool BIAS>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs a) {
    constexpr int W = vec<BF16>();
    __shared__ float sums[2 * kWaves];
    Lane<WIDE> at(a, sums);
    if (!WIDE && at.group >= a.groups) return;
    const int64_t base = (int64_t)at.group * a.size;
    const int64_t stride = WIDE ? a.strips : a.strips * kWaves;
    int64_t row = blockIdx.x / a.columns;
    if (!WIDE) row = row * kWaves + (threadIdx.x >> 6);
    Vec<BF16, WHOLE> w[NV], b[NV];
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int i = (at.first + m * at.lanes) * W;
        w[m].weights(a.weight, base, i, a.size, 1.f);
        if (BIAS) b[m].weights(a.bias, base, i, a.size, 0.f);
    }
    const int64_t width = (int64_t)a.groups * a.size;
    for (; row < a.rows; row += stride) {
        Vec<BF16, WHOLE> u[NV], z[NV];
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int i = (at.first + m * at.lanes) * W;
            u[m].ask(a.x, row * a.ldx + base, i, a.size);
            if (GATE) z[m].ask(a.z, row * a.ldz + base, i, a.size);
        }
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int i = (at.first + m * at.lanes) * W;
            u[m].take(i, a.size);
            if (GATE) z[m].take(i, a.size);
        }
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            if (GATE) {
#pragma unroll
                for (int e = 0; e < W; ++e) z[m].v[e] *= sigmoid(z[m].v[e]);
                if (GATE == kFirst)
#pragma unroll
                    for (int e = 0; e < W; ++e) u[m].v[e] *= z[m].v[e];
            }
        }
        normalise<BF16, NV, WIDE, WHOLE>(a, at, u);
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int i = (at.first + m * at.lanes) * W;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                u[m].v[e] *= w[m].v[e];
                if (BIAS) u[m].v[e] += b[m].v[e];
                if (GATE == kAfter) u[m].v[e] *= z[m].v[e];
            }
            u[m].store(a.y, row * width + base, i, a.size);
        }
    }
}

template <bool BF16, int NV, bool WIDE, bool WHOLE, int GATE, bool BIAS>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormArgs a) {
    constexpr int W = vec<BF16>();
    __shared__ float sums[2 * kWaves];
    __shared__ float joined[WIDE ? 1 : kWaves][WIDE ? 1 : 64 * NV * W];
    Lane<WIDE> at(a, sums);
    const bool mine = WIDE || at.group < a.groups;
    const int64_t base = (int64_t)at.group * a.size, width = (int64_t)a.groups * a.size;
    const int64_t strip = blockIdx.x / a.columns;
    const int64_t stride = WIDE ? a.strips : a.strips * kWaves;
    int64_t row = WIDE ? strip : strip * kWaves + (threadIdx.x >> 6);
    const float inv = 1.f / (float)a.size;
    Vec<BF16, WHOLE> w[NV], b[NV], dw[NV], db[NV];
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int i = (at.first + m * at.lanes) * W;
        if (mine) w[m].weights(a.weight, base, i, a.size, 1.f);
        if (BIAS && mine) b[m].weights(a.bias, base, i, a.size, 0.f);
#pragma unroll
        for (int e = 0; e < W; ++e) dw[m].v[e] = db[m].v[e] = 0.f;
    }
    for (; mine && row < a.rows; row += stride) {
        Vec<BF16, WHOLE> hat[NV], dy[NV], z[NV], x[NV];
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int i = (at.first + m * at.lanes) * W;
            x[m].ask(a.x, row * a.ldx + base, i, a.size);
            if (GATE) z[m].ask(a.z, row * a.ldz + base, i, a.size);
            dy[m].ask(a.dy, row * width + base, i, a.size);
        }
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int i = (at.first + m * at.lanes) * W;
            x[m].take(i, a.size);
            if (GATE) z[m].take(i, a.size);
            dy[m].take(i, a.size);
            hat[m] = x[m];
        }
        if (GATE == kFirst) {
#pragma unroll
            for (int m = 0; m < NV; ++m)
#pragma unroll
                for (int e = 0; e < W; ++e) hat[m].v[e] *= z[m].v[e] * sigmoid(z[m].v[e]);
        }
        const float factor = normalise<BF16, NV, WIDE, WHOLE>(a, at, hat);
        float s = 0.f, sh = 0.f;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                float d = dy[m].v[e];
                if (GATE == kAfter) {
                    const float zz = z[m].v[e], sg = sigmoid(zz), gate = zz * sg;
                    // d silu = sigmoid (1 + z (1 - sigmoid))
                    float pre = hat[m].v[e] * w[m].v[e];
                    if (BIAS) pre += b[m].v[e];
                    z[m].v[e] = d * pre * fmaf(gate, 1.f - sg, sg);
                    d *= gate;
                }
                dw[m].v[e] = fmaf(d, hat[m].v[e], dw[m].v[e]);
                if (BIAS) db[m].v[e] += d;
                d *= w[m].v[e];
                dy[m].v[e] = d;
                s += d;
                sh = fmaf(d, hat[m].v[e], sh);
            }
        }
        sh = at.sum(sh) * inv;
        s = a.center ? at.sum(s) * inv : 0.f;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int i = (at.first + m * at.lanes) * W;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                float d = (fmaf(-hat[m].v[e], sh, dy[m].v[e]) - s) * factor;
                if (GATE == kFirst) {
                    const float zz = z[m].v[e], sg = sigmoid(zz), gate = zz * sg;
                    z[m].v[e] = d * x[m].v[e] * fmaf(gate, 1.f - sg, sg);
                    d *= gate;
                }
                dy[m].v[e] = d;
            }
            dy[m].store(a.dx, row * width + base, i, a.size);
            if (GATE) z[m].store(a.dz, row * width + base, i, a.size);
        }
    }
    if (!a.part) return;
    float* out = a.part + strip * 2 * width;
    if constexpr (WIDE) {
#pragma unroll
        for (int m = 0; m < NV; ++m)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const int i = (at.first + m * at.lanes) * W + e;
                if (i < a.size) {
                    out[base + i] = dw[m].v[e];
                    if (BIAS) out[width + base + i] = db[m].v[e];
                }
            }
    } else {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int which = 0; which < (BIAS ? 2 : 1); ++which) {
            __syncthreads();
#pragma unroll
            for (int m = 0; m < NV; ++m)
#pragma unroll
                for (int e = 0; e < W; ++e)
                    joined[wave][(m * W + e) * 64 + lane] = which ? db[m].v[e] : dw[m].v[e];
            __syncthreads();
            // the lane's own channels again, a quarter of them for each wave
            if (mine)
                for (int x = wave; x < NV * W; x += kWaves) {
                    const int i = (at.first + x / W * at.lanes) * W + x % W, p = x * 64 + lane;
                    if (i < a.size)
                        out[which * width + base + i] = (joined[0][p] + joined[1][p]) +
                                                        (joined[2][p] + joined[3][p]);
                }
        }
    }
}

// dweight and dbias from the strips' sums: 16 channels a workgroup, whose 64 rows
// of lanes share the strips (64 channels and 16 rows left most of the chip idle:
// 1024 strips of 1536 channels 21 us).
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void norm_join_kernel(NormArgs a) {
    __shared__ float sums[kJoinWaves][16];
    const int64_t width = (int64_t)a.groups * a.size;
    const int which = blockIdx.y, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * 16 + (lane & 15);
    float* out = which ? a.dbias : a.dweight;
    if (!out) return;
    float s = 0.f;
    if (i < width)
#pragma unroll 4
        for (int64_t n = threadIdx.x >> 4; n < a.strips; n += kJoinWaves * 4)
            s += a.part[(n * 2 + which) * width + i];
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16) sums[wave][lane] = s;
    __syncthreads();
    if (threadIdx.x < 16 && i < width) {
        s = 0.f;
#pragma unroll
        for (int n = 0; n < kJoinWaves; ++n) s += sums[n][lane];
        out[i] = s;
    }
}

}  // namespace
}  // namespace norm

using namespace norm;

void norm_plan(NormArgs& a, bool bf16, bool backward) {
    const int units = (a.size + (bf16 ? 7 : 3)) / (bf16 ? 8 : 4);
    a.lanes = 1;
    while (a.lanes < 64 && a.lanes < units) a.lanes *= 2;
    if (units > 128) a.lanes = kThreads;  // more than 2 vectors of a wave's lanes
    const bool wide = a.lanes == kThreads;
    a.vecs = (units + a.lanes - 1) / a.lanes;
    a.columns = wide ? a.groups : (a.groups + 64 / a.lanes - 1) / (64 / a.lanes);
    // Workgroups that a CU holds side by side: weights are read, and partial sums
    // written, once for each.  (16384 x 1536 bf16 backward, one group: 768 of them
    // 110 us of a training pass, 1280 97, 2048 108; 5997 x 511 fp32, 7 groups: 1024
    // 32, 2048 28.)
    const int64_t all = backward && wide ? 1280 : 2048;
    const int64_t most = (all + a.columns - 1) / a.columns;
    const int64_t need = wide ? a.rows : (a.rows + kWaves - 1) / kWaves;
    a.strips = need < most ? need : most;
    if (a.strips < 1) a.strips = 1;
}

size_t norm_bwd_ws(const NormArgs& a) {
    return (size_t)a.strips * 2 * a.groups * a.size * sizeof(float);
}

int64_t norm_workgroups(const NormArgs& a) { return a.strips * a.columns; }

#define NORM_(kernel, B, L, G, S)                                                         \
    do {                                                                                  \
        if (a.lanes == kThreads) {                                                        \
            if (a.vecs == 1) kernel<B, 1, true, L, G, S><<<n, kThreads, 0, s>>>(a);       \
            else if (a.vecs == 2) kernel<B, 2, true, L, G, S><<<n, kThreads, 0, s>>>(a);  \
            else if (B || a.vecs <= 4)                                                    \
                kernel<B, 4, true, L, G, S><<<n, kThreads, 0, s>>>(a);                    \
            else kernel<false, 8, true, L, G, S><<<n, kThreads, 0, s>>>(a);               \
        } else if (a.vecs == 1) kernel<B, 1, false, L, G, S><<<n, kThreads, 0, s>>>(a);   \
        else kernel<B, 2, false, L, G, S><<<n, kThreads, 0, s>>>(a);                      \
    } while (0)
#define NORM_GATE_(kernel, B, L, S)                              \
    do {                                                         \
        if (!a.z) NORM_(kernel, B, L, kNone, S);                 \
        else if (a.gate_first) NORM_(kernel, B, L, kFirst, S);   \
        else NORM_(kernel, B, L, kAfter, S);                     \
    } while (0)
#define NORM_BIAS_(kernel, B)                                          \
    do {                                                               \
        const bool whole_ = a.size % vec<B>() == 0;                    \
        if (a.bias || a.dbias) {                                       \
            if (whole_) NORM_GATE_(kernel, B, true, true);             \
            else NORM_GATE_(kernel, B, false, true);                   \
        } else {                                                       \
            if (whole_) NORM_GATE_(kernel, B, true, false);            \
            else NORM_GATE_(kernel, B, false, false);                  \
        }                                                              \
    } while (0)

hipError_t launch_norm_fwd(const NormArgs& a, bool bf16, hipStream_t s) {
    ProfScope ps(s, kPhaseMain);
    const unsigned n = (unsigned)norm_workgroups(a);
    if (bf16) NORM_BIAS_(norm_fwd_kernel, true);
    else NORM_BIAS_(norm_fwd_kernel, false);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(NormArgs a, bool bf16, void* workspace, hipStream_t s) {
    const unsigned n = (unsigned)norm_workgroups(a);
    a.part = a.dweight || a.dbias ? (float*)workspace : nullptr;
    {
        ProfScope ps(s, kPhaseMain);
        if (bf16) NORM_BIAS_(norm_bwd_kernel, true);
        else NORM_BIAS_(norm_bwd_kernel, false);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    ProfScope ps(s, kPhaseReduce);
    const int64_t width = (int64_t)a.groups * a.size;
    norm_join_kernel<<<dim3((unsigned)((width + 15) / 16), a.dbias ? 2 : 1), 64 * kJoinWaves, 0,
                       s>>>(a);
    return hipGetLastError();
}
#undef NORM_BIAS_
#undef NORM_GATE_
#undef NORM_

}  // namespace msscan
