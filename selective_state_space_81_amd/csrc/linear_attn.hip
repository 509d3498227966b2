// linear_attn.hip -- linear attention with a decay for each head, forward:
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T      (S_{t-1} dropped where reset_t)
//   o_t = scale S_t^T q_t
//
// In blocks of tokens (linear_attn.h) all of it but the decays is products of
// small matrices, on the matrix cores.  A workgroup walks along the blocks of
// one (batch row, head, 64 columns of dv).  Four of its waves make a block's
// outputs, 16 queries each: their scores stay in registers, in the layout in
// which one matrix instruction leaves them and the next takes them (with the
// summed index permuted, which a sum allows), and their rows of q come straight
// from memory.  The other four move the state on, 16 columns each: [dk][16] in
// fp32, in registers, with a copy rounded to bf16 in LDS for the block's queries.
// Both need the state before the block only, so they run side by side.  Inputs
// are read once, the state never moves, and two barriers a block suffice.  Loads
// of the next block are under way while the present one is computed.
//
// A sequence is cut into segments where heads and columns are too few for the
// chip: a first pass sums up the segments but the last (k and v only), a second
// joins these, and the walk above starts from what they give.
//
// Bound by what a wave issues and waits for along its blocks, one after another
// (2.7 us each), with 1300 cycles of matrix instructions a wave in them: 8 x 2048
// tokens of 24 heads of 64 columns and shared keys of 128, 93 us; heads of 64 with
// keys of their own, states saved, 108 us; 131072 tokens of 12 heads of 128 x 128,
// 804 us, a third of them for the sums of segments.
#include <type_traits>

#include "linear_attn.h"
#include "msscan_internal.h"

namespace msscan {
namespace attn {
namespace {

// Workgroup -> columns (quickest), head, segment, batch row: heads that share
// q and k lie side by side, on one XCD.
struct Place {
    int tile, h, seg, b;
    __device__ __forceinline__ explicit Place(const AttnArgs& a, int nseg) {
        uint32_t id = xcd_logical(blockIdx.x, gridDim.x);
        tile = id % a.tiles, id /= a.tiles;
        h = id % a.H, id /= a.H;
        seg = id % nseg;
        b = id / nseg;
    }
};

// Tokens left, as far as a block goes.
__device__ __forceinline__ int there(int64_t n) { return n < 128 ? (int)n : 128; }

// A number that is the same again and again, but not to the compiler, which
// would keep a mask for every comparison with it.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// A wave's 16 columns of a state: tile t, entry r is S[16 t + 4 g + r][col].
template <int DK>
struct State {
    static constexpr int kTiles = DK / 16;
    f4 s[kTiles];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) s[t] = f4{0, 0, 0, 0};
    }
    // p: [dk][dv] of one head
    __device__ __forceinline__ void load(const float* p, int dk, int dv, int col) {
        const int row = (threadIdx.x & 63) >> 4 << 2;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = t * 16 + row + r;
                s[t][r] = d < dk && col < dv ? p[(int64_t)d * dv + col] : 0.f;
            }
    }
    __device__ __forceinline__ void store(float* p, int dk, int dv, int col) const {
        const int row = (threadIdx.x & 63) >> 4 << 2;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = t * 16 + row + r;
                if (d < dk && col < dv) p[(int64_t)d * dv + col] = s[t][r];
            }
    }
    // In whole tiles of 16 (a.DKs, a.DVs), the wave's first column vcol.
    __device__ __forceinline__ void keep(float* p, int dks, int dvs, int vcol) const {
        const int l = threadIdx.x & 63, row = l >> 4 << 2;
        if (vcol >= dvs) return;
        p += row * dvs + vcol + (l & 15);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            if (t * 16 < dks)
#pragma unroll
                for (int r = 0; r < 4; ++r) p[(t * 16 + r) * dvs] = s[t][r];
    }
    // The block's end: s = whole s + sum_j w_j x_j y_j^T, x in rows of xt, y in
    // rows of yt.  Nothing of a state before a document's start comes through.
    template <bool BF16, int XLD, int YLD, int kAtOnce, int N, class E>
    __device__ __forceinline__ void advance(const E* xt, const E* yt, int ycol, const Decays<N>& d,
                                            const float* w, float scale) {
        const bool cut = d.cut();
        const float whole = d.whole;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[t][r] = cut ? 0.f : s[t][r] * whole;
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int k0 = 0; k0 < N; k0 += 32) {
            f8 y = widen(across<YLD>(yt, k0, ycol));
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= w[k0 + g * 8 + e] * scale;
            const Parts<BF16> yp(y);
#pragma unroll
            for (int t0 = 0; t0 < kTiles; t0 += kAtOnce) {
                typename Io<BF16>::Frag xf[kAtOnce];
#pragma unroll
                for (int t = 0; t < kAtOnce; ++t) xf[t] = across<XLD>(xt, k0, (t0 + t) * 16);
#pragma unroll
                for (int n = Io<BF16>::kParts - 1; n >= 0; --n)
#pragma unroll
                    for (int t = 0; t < kAtOnce; ++t) s[t0 + t] = mma(xf[t], yp.p[n], s[t0 + t]);
            }
        }
    }
    // Rounded to the io type for the queries: [column][dk], this wave's columns.
    template <int LD, class E>
    __device__ __forceinline__ void publish(E* st, int vcol) const {
        const int l = threadIdx.x & 63;
        E* p = st + (vcol + (l & 15)) * LD + (l >> 4 << 2);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) put4(p + t * 16, s[t]);
    }
    // One token, where matrix products would carry what is not finite into
    // places that it does not reach: s = decay s + x y (keep false: s = x y).
    template <class E>
    __device__ __forceinline__ void token(const E* x, float y, float decay, bool keep, int dk) {
        const int row = (threadIdx.x & 63) >> 4 << 2;
        const int left = opaque(dk - row);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (t * 16 + r < left)
                    s[t][r] = fmaf(get(x + t * 16 + row + r), y, keep ? s[t][r] * decay : 0.f);
    }
    // q's product with the wave's columns, of one token
    template <class E>
    __device__ __forceinline__ float meet(const E* q, int dk) const {
        const int row = (threadIdx.x & 63) >> 4 << 2;
        const int left = opaque(dk - row);
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (t * 16 + r < left) sum = fmaf(get(q + t * 16 + row + r), s[t][r], sum);
        sum += __shfl_xor(sum, 16);
        return sum + __shfl_xor(sum, 32);
    }
};

// ---- forward ------------------------------------------------------------------------

// Eight waves: four make the block's outputs, four move the state on.  Both need
// the state before the block only, so they run side by side.
constexpr int kFwdThreads = 2 * kThreads;

// Two workgroups share a CU where dk is at most 64.  Above, a lone one has
// registers for everything; two (PAIR) keep 128 a wave, at the price of some that
// spill, of queries asked for late and of fewer tiles at once (one block a CU of
// 2.7 us against two of 5.1).
template <bool BF16, int DK, bool WHOLE, bool PAIR>
__global__ __launch_bounds__(kFwdThreads, DK == 64 || PAIR ? 4 : 2) void attn_fwd_kernel(AttnArgs a) {
    typedef typename Io<BF16>::E E;
    typedef typename Io<BF16>::Frag Frag;
    constexpr int N = Io<BF16>::kBlock, kIts = N / 16;  // tiles of queries, and of keys
    constexpr int kCols = 64 * kIts / kWaves;           // columns of a wave's outputs
    typedef Tile<BF16, DK, WHOLE, kFwdThreads> K;
    typedef Tile<BF16, 64, WHOLE, kFwdThreads> V;
    constexpr int SLD = DK + Io<BF16>::kPad;
    __shared__ __align__(16) E kt[K::kSize];
    __shared__ __align__(16) E vt[V::kSize];
    __shared__ __align__(16) E st[64 * SLD];  // the state before the block, [column][dk]
    __shared__ Decays<N> decays[2];
    __shared__ float glog[2][N];
    __shared__ int bad_block;  // the last one in which something was not finite

    const Place at(a, a.nseg);
    const int id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = id & 3;
    const bool outputs = id < kWaves;
    const int lane = threadIdx.x & 63, g = lane >> 4, s16 = lane & 15;
    const int col0 = at.tile * 64, vcol = wave * 16, mycol = col0 + vcol + s16;
    const int nv = a.dv - col0 < 64 ? a.dv - col0 : 64;
    const int kh = at.h / (a.H / a.Hk);
    const int64_t row0 = (int64_t)at.b * a.L;
    const E* q = (const E*)a.q + row0 * a.ldq + (int64_t)kh * a.dk;
    const E* k = (const E*)a.k + row0 * a.ldk + (int64_t)kh * a.dk;
    const E* v = (const E*)a.v + row0 * a.ldv + (int64_t)at.h * a.dv + col0;
    const int ldo = a.H * a.dv;
    const int blocks = (int)a.blocks;
    const int c0 = at.seg * (int)a.per, c1 = min(c0 + (int)a.per, blocks);
    const float scale = a.scale;
    const int64_t head = ((int64_t)at.b * a.H + at.h) * a.dk * a.dv;

    if (threadIdx.x == 0) bad_block = -1;
    lds_barrier();

    // Both roles load and store the tiles; wave 0, whose queries have the fewest
    // keys, sums the next block's decays up.
    K kr;
    V vr;
    Token tok;
    auto tokens = [&](int c) {  // of block c, at least one of which is there
        if (id == 0) tok.load(a, row0 + (int64_t)c * N, there(a.L - (int64_t)c * N), at.h, N);
    };
    auto settle = [&](int c) {
        if (id == 0) {
            tok.settle(there(a.L - (int64_t)c * N));
            decays[c & 1].make(tok.g, tok.reset);
            if (lane < N) glog[c & 1][lane] = tok.g;
        }
    };
    auto fetch = [&](int c) {
        const int64_t t0 = (int64_t)c * N;
        const int rows = there(a.L - t0);
        kr.load(k + t0 * a.ldk, (int)a.ldk, rows, a.dk);
        vr.load(v + t0 * a.ldv, (int)a.ldv, rows, nv);
    };
    // Tiles of block c in their places; whether it has to go token by token.
    auto stage = [&](int c) {
        const int rows = there(a.L - (int64_t)c * N);
        bool bad = kr.store(kt, rows, a.dk);
        bad |= vr.store(vt, rows, nv);
        if (bad) bad_block = c - c0;
        lds_barrier();
        if (c + 1 < c1) {
            settle(c + 1);
            if (c + 2 < c1) tokens(c + 2);
            fetch(c + 1);
        }
        return bad_block == c - c0;
    };
    tokens(c0);
    fetch(c0);
    settle(c0);
    if (c0 + 1 < c1) tokens(c0 + 1);

    if (!outputs) {
        State<DK> S;
        if (a.nseg > 1)
            S.load(a.seg + (((int64_t)at.b * a.nseg + at.seg) * a.H + at.h) * a.dk * a.dv, a.dk,
                   a.dv, mycol);
        else if (a.h0)
            S.load(a.h0 + head, a.dk, a.dv, mycol);
        else
            S.clear();
        for (int c = c0; c < c1; ++c) {
            S.template publish<SLD>(st, vcol);
            const bool slow = stage(c);
            const Decays<N>& dec = decays[c & 1];
            if (a.states)
                S.keep(a.states +
                           (((int64_t)at.b * a.blocks + c) * a.H + at.h) * a.DKs * (int64_t)a.DVs,
                       a.DKs, a.DVs, col0 + vcol);
            if (slow) {
                // token by token, outputs and all; the queries come where the
                // state's copy was
                const int64_t t0 = (int64_t)c * N;
                E* o = (E*)a.o + (row0 + t0) * ldo + (int64_t)at.h * a.dv + col0;
                lds_barrier();
                lds_barrier();
                for (int t = 0; t < min(there(a.L - t0), N); ++t) {
                    const bool starts = dec.start[t] == t;
                    S.token(kt + t * K::kLd, get(vt + t * V::kLd + vcol + s16),
                            hw_exp2(glog[c & 1][t] * kLog2e), !starts, a.dk);
                    const float sum = S.meet(st + t * SLD, a.dk);
                    if (g == 0 && vcol + s16 < nv)
                        dev::st<BF16>(o, t * ldo + vcol + s16, sum * scale);
                }
            } else {
                S.template advance<BF16, K::kLd, V::kLd, PAIR ? 2 : 4>(kt, vt, vcol, dec, dec.last, 1.f);
            }
            lds_barrier();
        }
        if (a.h_last && c1 == blocks) S.store(a.h_last + head, a.dk, a.dv, mycol);
        return;
    }

    const int it = wave % kIts, ocol = wave / kIts * kCols, i = it * 16 + s16;
    Rows<BF16, DK, WHOLE> qr;
    auto queries = [&](int c) {
        const int64_t t0 = (int64_t)c * N;
        qr.load(q + t0 * a.ldq, (int)a.ldq, it * 16, there(a.L - t0), a.dk);
    };
    queries(c0);
    for (int c = c0; c < c1; ++c) {
        const bool slow = stage(c);
        const Decays<N>& dec = decays[c & 1];
        const int64_t t0 = (int64_t)c * N;
        const int rows = there(a.L - t0);
        Frag qf[DK / 32];  // a query that is not finite stays in its own row
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) qf[s] = qr.operand(s, a.dk);
        if (!PAIR && c + 1 < c1) queries(c + 1);
        if (slow) {
            lds_barrier();
            if (id < kIts)
#pragma unroll
                for (int s = 0; s < DK / 32; ++s) put8(st + i * SLD + s * 32 + g * 8, qf[s]);
            lds_barrier();
            if (PAIR && c + 1 < c1) queries(c + 1);
            lds_barrier();
            continue;
        }
        // what the state before the block gives
        f4 oacc[kCols / 16];
#pragma unroll
        for (int n = 0; n < kCols / 16; ++n) oacc[n] = f4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < DK / 32; ++s)
#pragma unroll
            for (int n = 0; n < kCols / 16; ++n)
                oacc[n] = mma(along<SLD>(st, ocol + n * 16, s * 32), qf[s], oacc[n]);
        const int start = dec.start[i];
        const float first = dec.first[i] * scale;
#pragma unroll
        for (int n = 0; n < kCols / 16; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) oacc[n][r] = start < 0 ? oacc[n][r] * first : 0.f;
        // scores of 32 keys at a time, and what the keys' values give
        const float hi = dec.hi[i], lo = dec.lo[i];
        const int from = start < 0 ? 0 : start;
#pragma unroll
        for (int k0 = 0; k0 < N; k0 += 32) {
            if (k0 > it * 16) break;
            f4 p[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int s = 0; s < DK / 32; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    p[x] = mma(along<K::kLd>(kt, k0 + x * 16, s * 32), qf[s], p[x]);
            f8 w;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = k0 + x * 16 + g * 4;
                const f4 hj = *reinterpret_cast<const f4*>(&dec.hi[j]);
                const f4 lj = *reinterpret_cast<const f4*>(&dec.lo[j]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = (uint32_t)(j + r - from) <= (uint32_t)(i - from);
                    w[x * 4 + r] = only(in, p[x][r] * (decay(hi, lo, hj[r], lj[r]) * scale));
                }
            }
            const Frag pf = round(w, Frag{});
#pragma unroll
            for (int n = 0; n < kCols / 16; ++n)
                oacc[n] = mma(across_pair<V::kLd>(vt, k0, ocol + n * 16), pf, oacc[n]);
        }
        if (PAIR && c + 1 < c1) queries(c + 1);
        E* o = (E*)a.o + (row0 + t0) * ldo + (int64_t)at.h * a.dv + col0;
        if (i < rows)
#pragma unroll
            for (int n = 0; n < kCols / 16; ++n)
                store4<WHOLE>(o + i * ldo, ocol + n * 16 + g * 4, nv, oacc[n]);
        lds_barrier();
    }
}

// ---- walk of the states alone ----------------------------------------------------------
//
// Forward in time over (k, v), or backward over (scale q, dO), where the state
// is the gradient of the states: R before a block (in the walk's order) is dL/dS
// at the block's end, and a token's decay comes behind its own term.
template <bool BF16, int DK, bool WHOLE, bool REV, bool FULL>
__global__ __launch_bounds__(kThreads, DK == 64 ? 3 : 2) void attn_walk_kernel(AttnArgs a) {
    typedef typename Io<BF16>::E E;
    constexpr int N = Io<BF16>::kBlock;
    typedef Tile<BF16, DK, WHOLE> X;
    typedef Tile<BF16, 64, WHOLE> Y;
    __shared__ __align__(16) E xt[X::kSize];
    __shared__ __align__(16) E yt[Y::kSize];
    __shared__ Decays<N> decays[2];
    __shared__ float glog[2][N];
    __shared__ int bad_block;  // the last one in which something was not finite

    const Place at(a, FULL ? a.nseg : a.nseg - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, s16 = lane & 15;
    const int col0 = at.tile * 64, vcol = wave * 16, mycol = col0 + vcol + s16;
    const int nv = a.dv - col0 < 64 ? a.dv - col0 : 64;
    const int kh = at.h / (a.H / a.Hk);
    const int64_t row0 = (int64_t)at.b * a.L;
    const int64_t ldx = REV ? a.ldq : a.ldk, ldy = REV ? (int64_t)a.H * a.dv : a.ldv;
    const E* x = (const E*)(REV ? a.q : a.k) + row0 * ldx + (int64_t)kh * a.dk;
    const E* y = (const E*)(REV ? a.dO : a.v) + row0 * ldy + (int64_t)at.h * a.dv + col0;
    const float scale = REV ? a.scale : 1.f;
    const int blocks = (int)a.blocks;
    const int n0 = at.seg * (int)a.per, n1 = min(n0 + (int)a.per, blocks);
    const int64_t head = ((int64_t)at.b * a.H + at.h) * a.dk * a.dv;
    const int64_t seg = (((int64_t)at.b * a.nseg + at.seg) * a.H + at.h);
    const float* first = REV ? a.dh_last : a.h0;

    State<DK> S;
    S.clear();
    if (FULL) {
        if (a.nseg > 1)
            S.load(a.seg + seg * a.dk * a.dv, a.dk, a.dv, mycol);
        else if (first)
            S.load(first + head, a.dk, a.dv, mycol);
    }
    if (threadIdx.x == 0) bad_block = -1;

    double total = 0.0;  // of the segment's log decays, in base 2
    bool any = false;    // a document starts in it
    X xr;
    Y yr;
    Token tok;
    auto block = [&](int n) { return REV ? blocks - 1 - n : n; };
    auto tokens = [&](int n) {
        const int64_t t0 = (int64_t)block(n) * N;
        if (wave == 0) tok.load(a, row0 + t0, there(a.L - t0), at.h, N);
    };
    auto settle = [&](int n) {
        if (wave == 0) {
            tok.settle(there(a.L - (int64_t)block(n) * N));
            decays[n & 1].make(tok.g, tok.reset);
            if (lane < N) glog[n & 1][lane] = tok.g;
        }
    };
    auto fetch = [&](int n) {
        const int64_t t0 = (int64_t)block(n) * N;
        const int rows = there(a.L - t0);
        xr.load(x + t0 * ldx, (int)ldx, rows, a.dk);
        yr.load(y + t0 * ldy, (int)ldy, rows, nv);
    };
    tokens(n0);
    fetch(n0);
    settle(n0);
    if (n0 + 1 < n1) tokens(n0 + 1);
    lds_barrier();
    for (int n = n0; n < n1; ++n) {
        const int c = block(n);
        const int rows = there(a.L - (int64_t)c * N);
        bool bad = xr.store(xt, rows, a.dk);
        bad |= yr.store(yt, rows, nv);
        if (bad) bad_block = n - n0;
        lds_barrier();
        const Decays<N>& dec = decays[n & 1];
        if (n + 1 < n1) {
            settle(n + 1);
            if (n + 2 < n1) tokens(n + 2);
            fetch(n + 1);
        }
        if (FULL && REV)
            S.keep(a.grads + (((int64_t)at.b * a.blocks + c) * a.H + at.h) * a.DKs * (int64_t)a.DVs,
                   a.DKs, a.DVs, col0 + vcol);
        any |= dec.cut();
        total += (double)dec.hi[N - 1] + (double)dec.lo[N - 1];
        if (bad_block == n - n0) {
            const int m = min(rows, N);
            for (int e = 0; e < m; ++e) {
                const int t = REV ? m - 1 - e : e;
                const bool starts = dec.start[t] == t;
                const float decay = hw_exp2(glog[n & 1][t] * kLog2e);
                const float val = get(yt + t * Y::kLd + vcol + s16) * scale;
                if (REV) {
                    S.token(xt + t * X::kLd, val, 1.f, true, a.dk);
#pragma unroll
                    for (int i = 0; i < State<DK>::kTiles; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) S.s[i][r] = starts ? 0.f : S.s[i][r] * decay;
                } else {
                    S.token(xt + t * X::kLd, val, decay, !starts, a.dk);
                }
            }
        } else {
            S.template advance<BF16, X::kLd, Y::kLd, 4>(xt, yt, vcol, dec,
                                                     REV ? dec.first : dec.last, scale);
        }
        lds_barrier();
    }
    if (FULL) {
        if (REV && a.dh0 && n1 == blocks) S.store(a.dh0 + head, a.dk, a.dv, mycol);
    } else {
        S.store(a.seg + seg * a.dk * a.dv, a.dk, a.dv, mycol);
        if (at.tile == 0 && threadIdx.x == 0) a.seg_f[seg] = any ? -1.f : (float)exp2(total);
    }
}

// ---- joining the segments -------------------------------------------------------------
// In place: the sums of segments become the states before them, the first one's
// (h0) too, for h_last may take its place while the first segment is yet to start.
__global__ __launch_bounds__(kThreads) void attn_carry_kernel(AttnArgs a, const float* first) {
    const int64_t per = (int64_t)a.H * a.dk * a.dv, each = (int64_t)a.dk * a.dv;
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= per * a.batch) return;
    const int64_t b = e / per, i = e - b * per;
    float* p = a.seg + b * a.nseg * per + i;
    const float* f = a.seg_f + b * a.nseg * a.H + i / each;
    float s = first ? first[e] : 0.f;
    float own = p[0], decay = f[0];
    p[0] = s;
    for (int n = 0; n < a.nseg - 1; ++n) {
        const float next = n + 2 < a.nseg ? p[(n + 1) * per] : 0.f;
        const float fnext = n + 2 < a.nseg ? f[(int64_t)(n + 1) * a.H] : 0.f;
        s = decay < 0.f ? own : fmaf(decay, s, own);
        p[(n + 1) * per] = s;
        own = next, decay = fnext;
    }
}

// ---- steps -------------------------------------------------------------------------------
//
// A few tokens from a state that is read once (and written once): its bytes are
// all that counts.  A workgroup takes 64 columns of a head's state, a thread
// four columns of every 16th row, in registers; tokens' q, k, v and decays wait
// in LDS, BLOCK of them at a time.  The sums over rows are joined by two
// shuffles and, over the waves, through LDS, all tokens of a block at once.
// 256 sequences of 24 heads of 128 x 64: 74 us, 5.5 TB/s; 5 tokens of 32 such
// sequences without update 10 us, a launch and four trips to memory.
template <bool BF16, int BLOCK, bool WHOLE, bool PAST>
__global__ __launch_bounds__(kThreads) void attn_step_kernel(AttnArgs a) {
    constexpr int kRows = kMaxHeadDim / 16;
    __shared__ float qs[BLOCK][kMaxHeadDim], ks[BLOCK][kMaxHeadDim];
    __shared__ __align__(16) float vs[BLOCK][64];
    __shared__ __align__(16) float sums[BLOCK][kWaves][64];
    __shared__ float decay[BLOCK];

    const Place at(a, 1);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c = (threadIdx.x & 15) * 4, r0 = threadIdx.x >> 4;
    const int col0 = at.tile * 64, nv = a.dv - col0 < 64 ? a.dv - col0 : 64;
    const int kh = at.h / (a.H / a.Hk);
    const int T = (int)a.L;
    int count = T;
    if (a.counts) {
        count = a.counts[at.b];
        count = count < 0 ? 0 : count > T ? T : count;
    }
    if (count == 0) return;
    float* h = a.h + ((int64_t)at.b * a.H + at.h) * a.dk * a.dv + col0;
    // Loads ask for places that are there, without a branch, which would wait for
    // each; rows from dk on are not looked at, nor columns behind the last.
    f4 S[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        const float* p = h + (int64_t)min(m * 16 + r0, a.dk - 1) * a.dv;
        if constexpr (WHOLE) {
            const f4* from = reinterpret_cast<const f4*>(p + min(c, nv - 4));
            S[m] = PAST ? __builtin_nontemporal_load(from) : *from;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) S[m][e] = p[min(c + e, nv - 1)];
        }
    }
    const void* qp = a.q ? a.q : a.k;
    const int64_t ldq = a.q ? a.ldq : a.ldk;
    const int64_t row0 = (int64_t)at.b * T;
    for (int t0 = 0; t0 < count; t0 += BLOCK) {
        const int n = count - t0 < BLOCK ? count - t0 : BLOCK;
        if (t0) lds_barrier();
        // all loads ahead of what waits for them
        constexpr int kQk = (BLOCK * kMaxHeadDim + kThreads - 1) / kThreads;
        constexpr int kV = (BLOCK * 64 + kThreads - 1) / kThreads;
        float kv[kQk], qv[kQk], vv[kV];
#pragma unroll
        for (int m = 0; m < kQk; ++m) {
            const int i = m * kThreads + threadIdx.x, t = min(i / kMaxHeadDim, n - 1);
            const int d = min(i % kMaxHeadDim, a.dk - 1);
            const int64_t row = row0 + t0 + t;
            kv[m] = ld<BF16>(a.k, row * a.ldk + (int64_t)kh * a.dk + d);
            qv[m] = ld<BF16>(qp, row * ldq + (int64_t)kh * a.dk + d);
        }
#pragma unroll
        for (int m = 0; m < kV; ++m) {
            const int i = m * kThreads + threadIdx.x, t = min(i / 64, n - 1), d = min(i % 64, nv - 1);
            vv[m] = ld<BF16>(a.v, (row0 + t0 + t) * a.ldv + (int64_t)at.h * a.dv + col0 + d);
        }
        const float g = log_decay(a, row0 + t0 + min((int)threadIdx.x, n - 1), at.h);
#pragma unroll
        for (int m = 0; m < kQk; ++m) {
            const int i = m * kThreads + threadIdx.x;
            if (i < BLOCK * kMaxHeadDim) (&ks[0][0])[i] = kv[m], (&qs[0][0])[i] = qv[m];
        }
#pragma unroll
        for (int m = 0; m < kV; ++m) {
            const int i = m * kThreads + threadIdx.x;
            if (i < BLOCK * 64) (&vs[0][0])[i] = vv[m];
        }
        if ((int)threadIdx.x < n) {
            const float x = g * kLog2e;  // and what its rounding left
            const float rest = fmaf(g, kLog2e, -x) + g * 1.925963033500011079e-8f;
            decay[threadIdx.x] = g < kNoDecay ? -1.f : hw_exp2(x) * fmaf(rest, kLn2, 1.f);
        }
        lds_barrier();
        for (int t = 0; t < n; ++t) {
            const f4 v = *reinterpret_cast<const f4*>(&vs[t][c]);
            const float w = decay[t];
            f4 o = {0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < kRows; ++m) {
                const int d = m * 16 + r0;
                if (d >= a.dk) break;
                const float kd = ks[t][d];
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][e] = fmaf(kd, v[e], w < 0.f ? 0.f : S[m][e] * w);
                if (a.q) {
                    const float qd = qs[t][d];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = fmaf(qd, S[m][e], o[e]);
                }
            }
            if (!a.q) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] += __shfl_xor(o[e], 16);
                o[e] += __shfl_xor(o[e], 32);
            }
            if (lane < 16) *reinterpret_cast<f4*>(&sums[t][wave][c]) = o;
        }
        if (!a.q) continue;
        lds_barrier();
        for (int i = threadIdx.x; i < n * 64; i += kThreads) {
            const int t = i / 64, d = i % 64;
            const float sum = (sums[t][0][d] + sums[t][1][d]) + (sums[t][2][d] + sums[t][3][d]);
            if (d < nv)
                st<BF16>(a.o, ((row0 + t0 + t) * a.H + at.h) * a.dv + col0 + d, sum * a.scale);
        }
    }
    if (!a.update) return;
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        const int d = m * 16 + r0;
        if (d < a.dk) {
            float* p = h + (int64_t)d * a.dv + c;
            if constexpr (WHOLE) {
                if (c < nv) {
                    if (PAST) __builtin_nontemporal_store(S[m], reinterpret_cast<f4*>(p));
                    else *reinterpret_cast<f4*>(p) = S[m];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < nv) p[e] = S[m][e];
            }
        }
    }
}

// A kernel for the io type, dk's size, and rows of whole vectors or not.
#define ATTN_EACH_(do_, bf16, a)                            \
    do {                                                    \
        const bool whole_ = a.dk % 8 == 0 && a.dv % 8 == 0; \
        if (bf16 && a.dk <= 64) {                           \
            if (whole_) do_(true, 64, true);                \
            else do_(true, 64, false);                      \
        } else if (bf16) {                                  \
            if (whole_) do_(true, 128, true);               \
            else do_(true, 128, false);                     \
        } else if (a.dk <= 64) {                            \
            if (whole_) do_(false, 64, true);               \
            else do_(false, 64, false);                     \
        } else {                                            \
            if (whole_) do_(false, 128, true);              \
            else do_(false, 128, false);                    \
        }                                                   \
    } while (0)

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace attn

using namespace attn;

void attn_plan(AttnArgs& a, bool bf16) {
    const int64_t block = bf16 ? kAttnBlockBf16 : kAttnBlockF32;
    a.blocks = (a.L + block - 1) / block;
    a.tiles = (a.dv + 63) / 64;
    a.DKs = (a.dk + 15) / 16 * 16;
    a.DVs = (a.dv + 15) / 16 * 16;
    // Half a workgroup a CU and more walk the whole sequence: cut, they would pay
    // for the sums of segments.  Both sides, whole and cut (bf16, 64 x 64 of own keys
    // and 128 x 64 of shared ones, 2048 tokens): 96 workgroups 66 and 83 us, cut 50
    // and 68; 128 66 and 84, cut 52 and 73; 160 67 and 85, cut 65 and 89; 192 68,
    // cut 80; 240 86, cut 115.  The border is on the safe side: up to 160 a cut would
    // still win at 8192 tokens (327 and 403 us, cut 260 and 323), from 192 on never
    // (331, cut 359).  Fewer are cut until two a CU are there and none beyond them,
    // which would run by themselves at the end (131072 tokens of 12 heads of 128: 504
    // workgroups 805 us, 744 920); into segments of at least four blocks.
    const int64_t wgs = (int64_t)a.batch * a.H * a.tiles;
    int64_t nseg = wgs >= 128 ? 1 : 512 / wgs;
    if (nseg > a.blocks / 4) nseg = a.blocks / 4;
    if (nseg < 1) nseg = 1;
    a.per = (a.blocks + nseg - 1) / nseg;
    a.nseg = (int)((a.blocks + a.per - 1) / a.per);
}

AttnWs attn_ws(const AttnArgs& a, bool backward) {
    AttnWs w{};
    const size_t heads = (size_t)a.batch * a.H;
    size_t at = 0;
    w.seg = at;
    if (a.nseg > 1) at += up256(heads * a.nseg * a.dk * a.dv * sizeof(float));
    w.seg_f = at;
    if (a.nseg > 1) at += up256(heads * a.nseg * sizeof(float));
    w.grads = at;
    if (backward) at += up256(heads * a.blocks * a.DKs * a.DVs * sizeof(float));
    w.part = at;
    if (backward && a.fixed) at += up256(heads * a.blocks * sizeof(float));
    w.total = at;
    return w;
}

int64_t attn_workgroups(const AttnArgs& a, bool backward) {
    const int64_t walk = 2 * (int64_t)a.batch * a.H * a.tiles * a.nseg;  // of twice the threads
    const int64_t grad = backward ? (int64_t)a.batch * a.Hk * a.blocks : 0;
    const int64_t carry = ((int64_t)a.batch * a.H * a.dk * a.dv + kThreads - 1) / kThreads;
    const int64_t most = walk > grad ? walk : grad;
    return most > carry ? most : carry;
}

hipError_t launch_attn_carry(const AttnArgs& a, const float* first, hipStream_t s) {
    ProfScope ps(s, kPhaseCarry);
    const int64_t n = (int64_t)a.batch * a.H * a.dk * a.dv;
    attn_carry_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, first);
    return hipGetLastError();
}

hipError_t launch_attn_walk(const AttnArgs& a, bool bf16, bool reverse, bool full, hipStream_t s) {
    ProfScope ps(s, full ? kPhaseMain : kPhaseSummary);
    const unsigned n = (unsigned)((int64_t)a.batch * a.H * a.tiles * (full ? a.nseg : a.nseg - 1));
#define WALK_(B, DK, W)                                                                   \
    do {                                                                                  \
        if (!reverse)                                                                     \
            attn_walk_kernel<B, DK, W, false, false><<<n, kThreads, 0, s>>>(a);           \
        else if (full)                                                                    \
            attn_walk_kernel<B, DK, W, true, true><<<n, kThreads, 0, s>>>(a);             \
        else                                                                              \
            attn_walk_kernel<B, DK, W, true, false><<<n, kThreads, 0, s>>>(a);            \
    } while (0)
    ATTN_EACH_(WALK_, bf16, a);
#undef WALK_
    return hipGetLastError();
}

hipError_t launch_attn_fwd(AttnArgs a, bool bf16, void* workspace, hipStream_t s) {
    const AttnWs w = attn_ws(a, false);
    a.seg = (float*)((char*)workspace + w.seg);
    a.seg_f = (float*)((char*)workspace + w.seg_f);
    if (a.nseg > 1) {
        hipError_t e = launch_attn_walk(a, bf16, false, false, s);
        if (e != hipSuccess) return e;
        if ((e = launch_attn_carry(a, a.h0, s)) != hipSuccess) return e;
    }
    ProfScope ps(s, kPhaseMain);
    const unsigned n = (unsigned)((int64_t)a.batch * a.H * a.tiles * a.nseg);
#define FWD_(B, DK, W)                                                                \
    do {                                                                              \
        if (DK > 64 && n > 256) attn_fwd_kernel<B, DK, W, DK != 64><<<n, kFwdThreads, 0, s>>>(a); \
        else attn_fwd_kernel<B, DK, W, false><<<n, kFwdThreads, 0, s>>>(a);           \
    } while (0)
    ATTN_EACH_(FWD_, bf16, a);
#undef FWD_
    return hipGetLastError();
}

int64_t attn_step_workgroups(const AttnArgs& a) { return (int64_t)a.batch * a.H * a.tiles; }

hipError_t launch_attn_step(const AttnArgs& a, bool bf16, hipStream_t s) {
    ProfScope ps(s, kPhaseStep);
    // A large state goes past the caches: until the next step on it, the rest of a
    // model will have passed through them (256 sequences of 24 heads of 128 x 64,
    // 201 MB, several such in turn: 91 us against 101, before loads without branches
    // made it 74; one state by itself 80 against 74).
    const bool past = (double)a.batch * a.H * a.dk * a.dv * 4.0 > 64e6, whole = a.dv % 4 == 0;
    const unsigned n = (unsigned)attn_step_workgroups(a);
#define STEP_(B)                                                                       \
    do {                                                                               \
        if (a.L > 1) {                                                                 \
            if (whole) attn_step_kernel<B, 8, true, false><<<n, kThreads, 0, s>>>(a);  \
            else attn_step_kernel<B, 8, false, false><<<n, kThreads, 0, s>>>(a);       \
        } else if (!whole) {                                                           \
            attn_step_kernel<B, 1, false, false><<<n, kThreads, 0, s>>>(a);            \
        } else if (past) {                                                             \
            attn_step_kernel<B, 1, true, true><<<n, kThreads, 0, s>>>(a);              \
        } else {                                                                       \
            attn_step_kernel<B, 1, true, false><<<n, kThreads, 0, s>>>(a);             \
        }                                                                              \
    } while (0)
    if (bf16) STEP_(true);
    else STEP_(false);
#undef STEP_
    return hipGetLastError();
}

}  // namespace msscan
