// linear_attn_bwd.hip -- gradients of the linear attention.
//
// With R the gradient of the state at a block's end and S the state before the
// block, the block's gradients need nothing of other blocks.  With
//   A_ij = scale D_ij q_i . k_j       B_ij = scale D_ij dO_i . v_j
// (D the decays between tokens of one document, f and l those from the block's
// start and to its end, w the whole block's):
//   dv_j = sum_i A_ij dO_i + l_j R^T k_j
//   dq_i = sum_j B_ij k_j  + scale f_i S dO_i
//   dk_j = sum_i B_ij q_i  + l_j R v_j
//   dg_t = sum_{i >= t > j} A_ij dO_i . v_j + sum_{i >= t} scale f_i q_i . S dO_i
//          + sum_{j < t} l_j k_j . R v_j + w <R, S>
// The first sum of dg is a suffix sum, within the block and the document, of row
// sums less column sums: no cancellation over more than a block's tokens.
//
// The forward leaves S before each block (states); a walk backward in time
// (linear_attn.hip) leaves R (grads); then one workgroup a block and group of
// heads that share keys makes all gradients, adding those of q and k over the
// group's heads in registers, in their order: deterministic.
//
// 8 x 2048 tokens of 24 heads of 64 x 64 bf16: 152 us, 550 MB (both states are 200
// of them), and 72 for the walk.  Two workgroups a CU, each a chain of loads,
// scores, and products with the states' three parts; matrix instructions take a
// tenth of the time.  In fp32 with heads of 40 x 72, 3 x 1999 tokens of 6: 59 us.
#include <cstddef>
#include <type_traits>

#include "linear_attn.h"
#include "msscan_internal.h"

namespace msscan {
namespace attn {
namespace {

// Sums over the four lanes of the same l & 15, and over 16 neighbouring lanes, in
// every one of them, without trips through LDS.
__device__ __forceinline__ float sum_groups(float x) {
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t v = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
template <int CTRL>
__device__ __forceinline__ float turned(float x) {
    return __uint_as_float(
        __builtin_amdgcn_update_dpp(0u, __float_as_uint(x), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum_row(float x) {
    x += turned<0x128>(x);  // row_ror 8, 4, 2, 1
    x += turned<0x124>(x);
    x += turned<0x122>(x);
    return x + turned<0x121>(x);
}

template <bool BF16, int DK, int DV, bool WHOLE>
struct GradShared {
    typedef typename Io<BF16>::E E;
    static constexpr int N = Io<BF16>::kBlock, kIts = N / 16;
    static constexpr int kScoreLd = N + Io<BF16>::kPad, kStateLd = DV + Io<BF16>::kPad;
    __align__(16) E q[Tile<BF16, DK, WHOLE>::kSize];
    __align__(16) E k[Tile<BF16, DK, WHOLE>::kSize];
    __align__(16) E v[Tile<BF16, DV, WHOLE>::kSize];
    __align__(16) E dO[Tile<BF16, DV, WHOLE>::kSize];
    __align__(16) E A[N * kScoreLd];  // [i][j]
    __align__(16) E B[N * kScoreLd];
    __align__(16) E R[DK * kStateLd];  // rounded, for dv
    Decays<N> dec;
    float glog[N];
    int bad;  // number of the last head in which something was not finite
    float rows[kIts][N];  // [key tile][i]: sums of A_ij dO_i . v_j
    float cols[kIts][N];  // [query tile][j]
    float later[kWaves][N], earlier[kWaves][N], both[kWaves];
};

template <bool BF16, int DK, int DV, bool WHOLE>
__global__ __launch_bounds__(kThreads, DK + DV <= 128 ? 2 : 1) void attn_grad_kernel(AttnArgs a) {
    typedef typename Io<BF16>::E E;
    typedef typename Io<BF16>::Frag Frag;
    typedef GradShared<BF16, DK, DV, WHOLE> Shared;
    typedef Tile<BF16, DK, WHOLE> QK;
    typedef Tile<BF16, DV, WHOLE> V;
    constexpr int N = Shared::N, kIts = Shared::kIts, SLD = Shared::kScoreLd,
                  RLD = Shared::kStateLd, QLD = QK::kLd, VLD = V::kLd;
    constexpr int kKt = DK / 64, kVt = DV / 64;  // tiles of 16 channels a wave takes
    extern __shared__ __align__(16) char memory[];
    Shared& sh = *reinterpret_cast<Shared*>(memory);

    uint32_t id = xcd_logical(blockIdx.x, gridDim.x);
    const int kh = id % a.Hk;
    id /= a.Hk;
    const int64_t c = id % (uint32_t)a.blocks;
    const int b = id / (uint32_t)a.blocks;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, g = lane >> 4, s16 = lane & 15;
    const int group = a.H / a.Hk;
    const int64_t row0 = (int64_t)b * a.L + c * N;
    const int n = a.L - c * N < N ? (int)(a.L - c * N) : N, rows = n;

    // keys after queries; A and B lie side by side
    static_assert(offsetof(Shared, B) == offsetof(Shared, A) + sizeof sh.A &&
                      sizeof sh.A % sizeof(u4) == 0,
                  "one run of vectors");
    for (int i = threadIdx.x; i < (int)(2 * sizeof sh.A / sizeof(u4)); i += kThreads)
        reinterpret_cast<u4*>(sh.A)[i] = u4{0, 0, 0, 0};
    if (threadIdx.x == 0) sh.bad = 0;
    lds_barrier();

    f4 dq[kKt][kIts], dk[kKt][kIts];
#pragma unroll
    for (int m = 0; m < kKt; ++m)
#pragma unroll
        for (int it = 0; it < kIts; ++it) dq[m][it] = dk[m][it] = f4{0, 0, 0, 0};

    // Everything is asked for before the first wait; of a group's next head, v and
    // dO while the present one is worked on.
    V vr, dr;
    const int ldo = a.H * a.dv;
    auto fetch = [&](int h) {
        vr.load((const E*)a.v + row0 * a.ldv + (int64_t)h * a.dv, (int)a.ldv, rows, a.dv);
        dr.load((const E*)a.dO + row0 * ldo + (int64_t)h * a.dv, ldo, rows, a.dv);
    };
    Token tok;
    auto token = [&](int h) {
        if (wave == 0) tok.load(a, row0, rows, h, N);
    };
    token(kh * group);  // ahead of all else: its wave sums the decays up first
    bool qkbad;
    {
        QK qr, kr;
        qr.load((const E*)a.q + row0 * a.ldq + (int64_t)kh * a.dk, (int)a.ldq, rows, a.dk);
        kr.load((const E*)a.k + row0 * a.ldk + (int64_t)kh * a.dk, (int)a.ldk, rows, a.dk);
        fetch(kh * group);
        qkbad = qr.store(sh.q, rows, a.dk);
        qkbad |= kr.store(sh.k, rows, a.dk);
    }
    for (int n_head = 0; n_head < group; ++n_head) {
        const int h = kh * group + n_head;
        if (wave == 0) {
            tok.settle(rows);
            sh.dec.make(tok.g, tok.reset);
        }
        // tiles of the states as operands, on their way during the scores
        const int64_t at = (((int64_t)b * a.blocks + c) * a.H + h) * a.DKs * (int64_t)a.DVs;
        f8 sf[DV / 32], rf[DV / 32];
        auto states = [&](int m) {
            const int row = min((m * kWaves + wave) * 16 + s16, a.DKs - 1) * a.DVs;
#pragma unroll
            for (int e = 0; e < DV / 32; ++e) {
                const int p = row + min(e * 32 + g * 8, a.DVs - 8);
                sf[e] = *reinterpret_cast<const f8_align16*>(a.states + at + p);
                rf[e] = *reinterpret_cast<const f8_align16*>(a.grads + at + p);
            }
        };
        states(0);
        bool bad = qkbad;
        bad |= vr.store(sh.v, rows, a.dv);
        bad |= dr.store(sh.dO, rows, a.dv);
        if (bad) sh.bad = n_head + 1;
        lds_barrier();
        const bool slow = sh.bad == n_head + 1;
        const Decays<N>& dec = sh.dec;
        if (n_head + 1 < group) {
            token(h + 1);
            fetch(h + 1);
        }

        // scores, and the sums over them that the decays' gradient needs
#pragma unroll
        for (int m = 0; m < (kIts * (kIts + 1) / 2 + kWaves - 1) / kWaves; ++m) {
            int it = 0, jt = m * kWaves + wave;
            while (jt > it) jt -= ++it;
            if (it >= kIts) break;
            f4 qk = {0, 0, 0, 0}, ov = {0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < DK; d += 32)
                qk = mma(along<QLD>(sh.k, jt * 16, d), along<QLD>(sh.q, it * 16, d), qk);
#pragma unroll
            for (int d = 0; d < DV; d += 32)
                ov = mma(along<VLD>(sh.v, jt * 16, d), along<VLD>(sh.dO, it * 16, d), ov);
            const int i = it * 16 + s16, j = jt * 16 + g * 4;
            const float hi = dec.hi[i], lo = dec.lo[i];
            const int start = dec.start[i], from = start < 0 ? 0 : start;
            const f4 hj = *reinterpret_cast<const f4*>(&dec.hi[j]);
            const f4 lj = *reinterpret_cast<const f4*>(&dec.lo[j]);
            f4 A, B, M;
            float row = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = (uint32_t)(j + r - from) <= (uint32_t)(i - from);
                const float w = a.scale * decay(hi, lo, hj[r], lj[r]);
                A[r] = only(in, qk[r] * w);
                B[r] = only(in, ov[r] * w);
                M[r] = only(in, A[r] * ov[r]);
                row += M[r];
                const float col = sum_row(M[r]);
                if (s16 == 0) sh.cols[it][j + r] = col;
            }
            row = sum_groups(row);
            if (g == 0) sh.rows[jt][i] = row;
            put4(sh.A + i * SLD + j, A);
            put4(sh.B + i * SLD + j, B);
        }
        // dq and dk: what other blocks give
        f4 dqs[kIts], dks[kIts];
        float later[kIts], earlier[kIts], both = 0.f;
#pragma unroll
        for (int it = 0; it < kIts; ++it) later[it] = earlier[it] = 0.f;
#pragma unroll
        for (int m = 0; m < kKt; ++m) {
            const int d0 = (m * kWaves + wave) * 16;
#pragma unroll
            for (int it = 0; it < kIts; ++it) dqs[it] = dks[it] = f4{0, 0, 0, 0};
            if (m) states(m);
#pragma unroll
            for (int e0 = 0; e0 < DV; e0 += 32) {
                const int e = e0 + g * 8;
                f8 s = sf[e0 / 32], r = rf[e0 / 32];
                const bool in = d0 < a.DKs && e < a.DVs;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    s[x] = in ? s[x] : 0.f;
                    r[x] = in ? r[x] : 0.f;
                    both = fmaf(s[x], r[x], both);
                }
                const Parts<BF16> sp(s), rp(r);
                put8(sh.R + (d0 + s16) * RLD + e, rp.p[0]);
#pragma unroll
                for (int it = 0; it < kIts; ++it) {
                    dqs[it] = sp.times(along<VLD>(sh.dO, it * 16, e0), dqs[it]);
                    dks[it] = rp.times(along<VLD>(sh.v, it * 16, e0), dks[it]);
                }
            }
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int i = it * 16 + s16;
                const bool before = dec.start[i] < 0, after = i >= dec.start[N - 1];
                const float f = dec.first[i] * a.scale, l = dec.last[i];
                const f4 qi = get4(sh.q + i * QLD + d0 + g * 4);
                const f4 ki = get4(sh.k + i * QLD + d0 + g * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = before ? dqs[it][r] * f : 0.f;
                    const float y = after ? dks[it][r] * l : 0.f;
                    dq[m][it][r] += x;
                    dk[m][it][r] += y;
                    later[it] += before ? qi[r] * x : 0.f;
                    earlier[it] += after ? ki[r] * y : 0.f;
                }
            }
        }
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
            later[it] = sum_groups(later[it]);
            earlier[it] = sum_groups(earlier[it]);
            if (g == 0) {
                sh.later[wave][it * 16 + s16] = later[it];
                sh.earlier[wave][it * 16 + s16] = earlier[it];
            }
        }
        both = sum_groups(sum_row(both));
        if (lane == 0) sh.both[wave] = both;
        lds_barrier();

        // within the block
        f4 dv[kVt][kIts];
#pragma unroll
        for (int m = 0; m < kVt; ++m)
#pragma unroll
            for (int jt = 0; jt < kIts; ++jt) dv[m][jt] = f4{0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < kVt; ++m) {
            const int e0 = (m * kWaves + wave) * 16;
#pragma unroll
            for (int d = 0; d < DK; d += 32) {
                const Frag rf = across<RLD>(sh.R, d, e0);
#pragma unroll
                for (int jt = 0; jt < kIts; ++jt)
                    dv[m][jt] = mma(rf, along<QLD>(sh.k, jt * 16, d), dv[m][jt]);
            }
#pragma unroll
            for (int jt = 0; jt < kIts; ++jt) {
                const int j = jt * 16 + s16;
                const bool after = j >= dec.start[N - 1];
                const float l = dec.last[j];
#pragma unroll
                for (int r = 0; r < 4; ++r) dv[m][jt][r] = after ? dv[m][jt][r] * l : 0.f;
            }
        }
        if (!slow) {
#pragma unroll
            for (int k0 = 0; k0 < N; k0 += 32) {
#pragma unroll
                for (int m = 0; m < kKt; ++m) {
                    const int d0 = (m * kWaves + wave) * 16;
                    const Frag kf = across<QLD>(sh.k, k0, d0), qf = across<QLD>(sh.q, k0, d0);
#pragma unroll
                    for (int it = k0 / 16; it < kIts; ++it)
                        dq[m][it] = mma(kf, along<SLD>(sh.B, it * 16, k0), dq[m][it]);
#pragma unroll
                    for (int jt = 0; jt < k0 / 16 + 2; ++jt)
                        dk[m][jt] = mma(qf, across<SLD>(sh.B, k0, jt * 16), dk[m][jt]);
                }
#pragma unroll
                for (int m = 0; m < kVt; ++m) {
                    const Frag of = across<VLD>(sh.dO, k0, (m * kWaves + wave) * 16);
#pragma unroll
                    for (int jt = 0; jt < k0 / 16 + 2; ++jt)
                        dv[m][jt] = mma(of, across<SLD>(sh.A, k0, jt * 16), dv[m][jt]);
                }
            }
        } else {
            // something is not finite: only the pairs of tokens that there are
            for (int x = 0; x < n; ++x) {
#pragma unroll
                for (int it = 0; it < kIts; ++it) {
                    const int i = it * 16 + s16;
                    const bool to = x <= i && x >= dec.start[i] && i < n;
                    const bool from = i <= x && i >= dec.start[x];
#pragma unroll
                    for (int m = 0; m < kKt; ++m) {
                        const int d0 = (m * kWaves + wave) * 16 + g * 4;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (to)
                                dq[m][it][r] = fmaf(get(sh.B + i * SLD + x),
                                                    get(sh.k + x * QLD + d0 + r), dq[m][it][r]);
                            if (from)
                                dk[m][it][r] = fmaf(get(sh.B + x * SLD + i),
                                                    get(sh.q + x * QLD + d0 + r), dk[m][it][r]);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < kVt; ++m) {
                        const int e0 = (m * kWaves + wave) * 16 + g * 4;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (from)
                                dv[m][it][r] = fmaf(get(sh.A + x * SLD + i),
                                                    get(sh.dO + x * VLD + e0 + r), dv[m][it][r]);
                    }
                }
            }
        }
        E* out = (E*)a.dv_out + row0 * a.H * a.dv + (int64_t)h * a.dv;
#pragma unroll
        for (int m = 0; m < kVt; ++m)
#pragma unroll
            for (int jt = 0; jt < kIts; ++jt) {
                const int j = jt * 16 + s16;
                if (j < n)
                    store4<WHOLE>(out + j * ldo, (m * kWaves + wave) * 16 + g * 4, a.dv,
                           dv[m][jt]);
            }
        // the decays
        if (slow) {
            // the pairs that straddle each token, by themselves: sums over rows and
            // columns would carry a NaN to tokens that it does not reach
            for (int t = wave; t < n; t += kWaves) {
                float sum = 0.f;
                if (lane >= t && lane < n) {
                    const int i = lane, start = dec.start[i];
                    for (int j = start < 0 ? 0 : start; j < t; ++j) {
                        float qk = 0.f, ov = 0.f;
                        for (int d = 0; d < a.dk; ++d)
                            qk = fmaf(get(sh.q + i * QLD + d), get(sh.k + j * QLD + d), qk);
                        for (int d = 0; d < a.dv; ++d)
                            ov = fmaf(get(sh.dO + i * VLD + d), get(sh.v + j * VLD + d), ov);
                        sum += qk * ov * a.scale *
                               decay(dec.hi[i], dec.lo[i], dec.hi[j], dec.lo[j]);
                    }
                }
                sum = sum_groups(sum_row(sum));
                if (lane == 0) sh.glog[t] = sum;
            }
            lds_barrier();
        }
        if (wave == 0) {
            const int t = lane < N ? lane : N - 1;
            float net = 0.f, late = 0.f, early = 0.f;
            if (lane < n) {
                if (!slow) {
                    for (int x = 0; x <= t / 16; ++x) net += sh.rows[x][t];
                    for (int x = t / 16; x < kIts; ++x) net -= sh.cols[x][t];
                }
                late = sh.later[0][t] + sh.later[1][t] + sh.later[2][t] + sh.later[3][t];
                early = sh.earlier[0][t] + sh.earlier[1][t] + sh.earlier[2][t] + sh.earlier[3][t];
            }
            net += late;
            // a document's tokens lie side by side and share its start
            const int start = dec.start[t];
#pragma unroll
            for (int d = 1; d < N; d *= 2) {
                const float x = __shfl_down(net, d), y = __shfl_up(early, d);
                const int theirs = __shfl_down(start, d);
                if (lane + d < N && theirs == start) net += x;
                if (lane >= d) early += y;
            }
            early = __shfl_up(early, 1);
            if (lane == 0) early = 0.f;
            const float rs = dec.cut() ? 0.f
                                       : dec.whole * ((sh.both[0] + sh.both[1]) +
                                                      (sh.both[2] + sh.both[3]));
            float dg = net + early + rs;
            if (slow && lane < n) dg += sh.glog[lane];
            if (start == t || lane >= n) dg = 0.f;
            if (a.fixed) {
                dg = sum_groups(sum_row(dg));
                if (lane == 0) a.part[((int64_t)b * a.blocks + c) * a.H + h] = dg;
            } else if (lane < n) {
                a.dg[(row0 + lane) * a.H + h] = dg;
            }
        }
        if (n_head + 1 < group) lds_barrier();
    }
    const int ldqk = a.Hk * a.dk;
    E* oq = (E*)a.dq + row0 * ldqk + (int64_t)kh * a.dk;
    E* ok = (E*)a.dk_out + row0 * ldqk + (int64_t)kh * a.dk;
#pragma unroll
    for (int m = 0; m < kKt; ++m)
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
            const int i = it * 16 + s16, d0 = (m * kWaves + wave) * 16 + g * 4;
            if (i < n) {
                store4<WHOLE>(oq + i * ldqk, d0, a.dk, dq[m][it]);
                store4<WHOLE>(ok + i * ldqk, d0, a.dk, dk[m][it]);
            }
        }
}

// Gradient of decays that are fixed for a head: the blocks' sums, in order
// within a thread and then as a tree.
__global__ __launch_bounds__(kThreads) void attn_fixed_kernel(AttnArgs a) {
    __shared__ double sums[kThreads];
    const int h = blockIdx.x;
    const int64_t n = a.batch * a.blocks;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += (double)a.part[i * a.H + h];
    sums[threadIdx.x] = s;
    lds_barrier();
    for (int d = kThreads / 2; d; d /= 2) {
        if ((int)threadIdx.x < d) sums[threadIdx.x] += sums[threadIdx.x + d];
        lds_barrier();
    }
    if (threadIdx.x == 0) a.dg[h] = (float)sums[0];
}

template <bool BF16, int DK, int DV, bool WHOLE>
hipError_t launch_grad(const AttnArgs& a, hipStream_t s) {
    constexpr int bytes = (int)sizeof(GradShared<BF16, DK, DV, WHOLE>);
    static_assert(bytes <= 160 * 1024, "LDS of a CU");
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(attn_grad_kernel<BF16, DK, DV, WHOLE>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const unsigned n = (unsigned)((int64_t)a.batch * a.Hk * a.blocks);
    attn_grad_kernel<BF16, DK, DV, WHOLE><<<n, kThreads, bytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

using namespace attn;

hipError_t launch_attn_bwd(AttnArgs a, bool bf16, void* workspace, hipStream_t s) {
    const AttnWs w = attn_ws(a, true);
    a.seg = (float*)((char*)workspace + w.seg);
    a.seg_f = (float*)((char*)workspace + w.seg_f);
    a.grads = (float*)((char*)workspace + w.grads);
    a.part = (float*)((char*)workspace + w.part);
    hipError_t e;
    if (a.nseg > 1) {
        if ((e = launch_attn_walk(a, bf16, true, false, s)) != hipSuccess) return e;
        if ((e = launch_attn_carry(a, a.dh_last, s)) != hipSuccess) return e;
    }
    if ((e = launch_attn_walk(a, bf16, true, true, s)) != hipSuccess) return e;
    {
        ProfScope ps(s, kPhaseMain);
#define GRAD_(B, W)                                                     \
    (a.dk <= 64 ? a.dv <= 64 ? launch_grad<B, 64, 64, W>(a, s)          \
                             : launch_grad<B, 64, 128, W>(a, s)         \
                : a.dv <= 64 ? launch_grad<B, 128, 64, W>(a, s)         \
                             : launch_grad<B, 128, 128, W>(a, s))
        if (a.dk % 8 == 0 && a.dv % 8 == 0) e = bf16 ? GRAD_(true, true) : GRAD_(false, true);
        else e = bf16 ? GRAD_(true, false) : GRAD_(false, false);
#undef GRAD_
        if (e != hipSuccess) return e;
    }
    if (a.fixed) {
        ProfScope ps(s, kPhaseReduce);
        attn_fixed_kernel<<<a.H, kThreads, 0, s>>>(a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace msscan
