// The notes of the token log probabilities' forward (logprob_notes.h) on the
// CPU: a row's blocks go through them wave by wave, as the kernel takes them,
// with the 64 lanes as contexts that meet at each ballot.  Checks that nothing
// is written outside the notes' room and that the alternatives found by reading
// the noted blocks again are the row's.
//
// Exits 0, or prints each failing case and exits 1.
#define __device__
#define __forceinline__ inline

#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <string>
#include <utility>
#include <vector>

// As on the device: of a NaN, signalling or not, and a number the number.
static float device_max(float a, float b) { return a != a ? b : b != b ? a : a > b ? a : b; }
#define fmaxf device_max

#include "logprob_notes.h"

using namespace msscan;

namespace {

// ---- 64 lanes that run in turn and meet at each ballot ----------------------
struct Lanes {
    static constexpr size_t kStack = 64 << 10;
    ucontext_t home, at[64];
    std::vector<char> stack = std::vector<char>(64 * kStack);
    std::function<void(int)> body;
    int now = 0;
    bool done[64];
    uint64_t votes[2];
    uint32_t round[64];

    void run(std::function<void(int)> f);
    void pass() { swapcontext(&at[now], &home); }
};
Lanes* lanes;

void lane_main() {
    lanes->body(lanes->now);
    lanes->done[lanes->now] = true;
    lanes->pass();
}

void Lanes::run(std::function<void(int)> f) {
    body = std::move(f);
    votes[0] = votes[1] = 0;
    for (int l = 0; l < 64; ++l) {
        done[l] = false;
        round[l] = 0;
        getcontext(&at[l]);
        at[l].uc_stack.ss_sp = stack.data() + l * kStack;
        at[l].uc_stack.ss_size = kStack;
        at[l].uc_link = &home;
        makecontext(&at[l], lane_main, 0);
    }
    while (!done[63]) {
        for (now = 0; now < 64; ++now) swapcontext(&home, &at[now]);
    }
    for (int l = 0; l < 64; ++l)
        if (!done[l] || round[l] != round[0]) {
            printf("lanes went apart\n");
            exit(1);
        }
}

struct Wave {
    static uint64_t ballot(bool v) {
        const uint32_t r = lanes->round[lanes->now]++ & 1;
        if (lanes->now == 0) lanes->votes[r] = 0;
        lanes->votes[r] |= (uint64_t)v << lanes->now;
        lanes->pass();
        return lanes->votes[r];
    }
    static void sync() { ballot(false); }
};

// ---- the kernel's way through a row --------------------------------------------
const float kInf = __builtin_inff();

// Threshold::take: the top-th largest of the maxima of neighbouring lanes.
float threshold(const std::vector<float>& lane_max, int top, int waves) {
    int shift = top <= 8 ? 3 : top <= 16 ? 2 : top <= 32 ? 1 : 0;
    if (waves == 16) shift = std::min(shift + 2, 4);
    std::vector<float> g;
    for (size_t k = 0; k < lane_max.size(); k += 1u << shift)
        g.push_back(*std::max_element(lane_max.begin() + k, lane_max.begin() + k + (1 << shift)));
    std::sort(g.begin(), g.end(), std::greater<float>());
    return g[top - 1];
}

struct Guarded {
    Notes notes;
    uint32_t after[512];
};

// `N` logits a vector, two vectors a lane and block, `W` waves.
bool check(const std::string& name, const std::vector<float>& x, int N, int W, int top) {
    const uint32_t V = (uint32_t)x.size(), nvec = V / N;
    auto fail = [&](const char* what) {
        printf("%s, %u logits of %d a vector, %d waves, top %d: %s\n", name.c_str(), V, N, W, top, what);
        return false;
    };
    auto block_max = [&](uint32_t b, int lane) {
        float m = -kInf;
        for (int u = 0; u < 2; ++u) {
            const uint32_t vec = b + u * 64 + lane;
            for (int e = 0; vec < nvec && e < N; ++e) m = fmaxf(m, x[vec * N + e]);
        }
        return m;
    };
    std::vector<float> first(64 * W, -kInf), all(64 * W, -kInf);
    for (int w = 0; w < W; ++w)
        for (int l = 0; l < 64; ++l)
            if ((uint32_t)w * 128 < nvec) first[w * 64 + l] = block_max(w * 128, l);
    const float thr = threshold(first, top, W);
    std::vector<Guarded> g(W);
    std::vector<int> count(W);
    std::vector<float> bound(W);
    bool past = false;
    for (int w = 0; w < W; ++w) {
        for (uint32_t& v : g[w].after) v = 0xabcdabcd;
        lanes->run([&](int lane) {
            Noted<Wave> n;
            n.init(&g[w].notes, top, lane);
            n.thr = n.bound = thr;
            auto take = [&](bool any, uint32_t token, float mb) {
                const bool in = any && mb >= n.thr;
                if (Wave::ballot(in)) n.note(in, token, mb);
                if (n.count > kNoteRoom) past = true;
                all[w * 64 + lane] = fmaxf(all[w * 64 + lane], mb);
            };
            for (uint32_t b = w * 128; b < nvec; b += 128 * W)
                take(b + lane < nvec, (b + lane) * N, block_max(b, lane));
            if (w == 0 && nvec * N < V) {
                const uint32_t i = nvec * N + lane;
                take(i < V, i, i < V ? x[i] : -kInf);
            }
            if (lane == 0) count[w] = n.count, bound[w] = n.bound;
        });
        for (uint32_t v : g[w].after)
            if (past || v != 0xabcdabcd) return fail("written outside the notes");
    }
    float t = threshold(all, top, W);
    for (float b : bound) t = fmaxf(t, b);
    typedef std::pair<float, uint32_t> Entry;
    auto before = [](const Entry& a, const Entry& b) {
        return a.first != b.first ? a.first > b.first : a.second < b.second;
    };
    std::vector<Entry> got, want;
    for (int w = 0; w < W; ++w)
        for (int k = 0; k < count[w]; ++k) {
            const uint32_t from = g[w].notes.first[k];
            if (from >= V) return fail("a noted token is outside the row");
            for (int e = 0; e < 2 * N; ++e) {
                const uint32_t tok = from < nvec * N ? from + e / N * (64 * N) + e % N : from + e;
                const bool have = from < nvec * N ? tok < nvec * N : e == 0;
                if (have && x[tok] >= t) got.push_back({x[tok], tok});
            }
        }
    for (uint32_t k = 0; k < V; ++k)
        if (x[k] == x[k]) want.push_back({x[k], k});
    std::sort(got.begin(), got.end(), before);
    std::sort(want.begin(), want.end(), before);
    if ((int)got.size() < top) return fail("alternatives lost");
    for (int k = 0; k < top; ++k)
        if (got[k] != want[k]) return fail("other alternatives than the row's");
    return true;
}

}  // namespace

int main() {
    lanes = new Lanes;
    bool ok = true;
    struct Size {
        uint32_t V;
        int N, W;
    };
    for (const Size s : {Size{50280, 8, 4}, Size{10500, 4, 4}, Size{131072, 8, 16}, Size{70001, 4, 16}}) {
        std::vector<std::pair<std::string, std::vector<float>>> rows;
        auto row = [&](const char* name, auto f) {
            std::vector<float> x(s.V);
            for (uint32_t k = 0; k < s.V; ++k) x[k] = f(k);
            rows.emplace_back(name, std::move(x));
        };
        uint32_t seed = 12345;
        auto random = [&] {
            seed = seed * 1664525u + 1013904223u;
            return (float)(seed >> 8) * 0x1p-24f;
        };
        row("all +inf", [](uint32_t) { return kInf; });
        row("every other +inf", [](uint32_t k) { return k % 2 ? kInf : (float)(k % 97); });
        row("every 16th +inf", [](uint32_t k) { return k % 16 == 5 ? kInf : -1.f; });
        row("rising, then +inf", [&](uint32_t k) { return k > s.V / 2 ? kInf : (float)k; });
        row("+inf at the end", [&](uint32_t k) { return k > s.V - 3 ? kInf : 0.f; });
        row("a third +inf, a third NaN", [&](uint32_t) {
            const float v = random();
            return v < 0.33f ? kInf : v < 0.66f ? __builtin_nanf("") : v;
        });
        row("rising", [](uint32_t k) { return (float)k; });
        row("all -inf", [](uint32_t) { return -kInf; });
        row("all 3e38", [](uint32_t) { return 3e38f; });
        row("random", [&](uint32_t) { return random() - 0.5f; });
        for (const auto& r : rows)
            for (const int top : {1, 5, 64}) ok = check(r.first, r.second, s.N, s.W, top) && ok;
    }
    return ok ? 0 : 1;
}
