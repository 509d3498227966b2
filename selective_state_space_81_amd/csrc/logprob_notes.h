// logprob_notes.h -- the blocks of logits that a wave of the token log
// probabilities' forward notes for its alternatives (logprob.hip).  Free of
// HIP's own functions, so that a host test can run it: `Wave` is the wave.
#pragma once

#include <math.h>
#include <stdint.h>

namespace msscan {
namespace {

__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float float_of(uint32_t b) { return __builtin_bit_cast(float, b); }

// The smallest float above v < infinity (x > v is then x >= next for every fp32 x).
__device__ __forceinline__ float next_above(float v) {
    const uint32_t b = bits_of(v + 0.f);
    return float_of((b >> 31) ? b - 1 : b + 1);
}

// Blocks that a wave has noted, in LDS: the first token and the largest logit
// of each.  kNoteRoom: what is kept of a flush (below) is at most what came
// together since the one before (kNoteFlush and a block of 64 lanes) and fewer
// than `top` (64) more, and another block may follow.
constexpr int kNoteFlush = 128, kNoteRoom = kNoteFlush + 64 + 64 + 64;
struct Notes {
    uint32_t first[kNoteRoom];
    float high[kNoteRoom];
};

template <class Wave>
struct Noted {
    Notes* q;
    float thr;    // what a block's largest logit has to reach to be noted (NaN: none does)
    float bound;  // what at least `top` logits of the row reach
    int top, count, lane;

    __device__ __forceinline__ void init(Notes* notes, int top_, int lane_) {
        q = notes;
        thr = bound = -__builtin_inff();
        top = top_;
        count = 0;
        lane = lane_;
    }
    __device__ __forceinline__ void note(bool in, uint32_t first, float high) {
        const uint64_t m = Wave::ballot(in);
        const int k = count + __builtin_popcountll(m & ((1ull << lane) - 1));
        if (in && k < kNoteRoom) {  // never past it, see kNoteRoom
            q->first[k] = first;
            q->high[k] = high;
        }
        count += __builtin_popcountll(m);
        count = count < kNoteRoom ? count : kNoteRoom;
        if (count >= kNoteFlush) flush();
    }
    // Many notes (rows that rise): the top-th largest of their maxima is reached
    // by `top` logits, so notes below it go.  Blocks to come have higher tokens
    // and have to exceed it; nothing exceeds +infinity.
    __device__ __forceinline__ void flush() {
        constexpr int K = kNoteRoom / 64;
        Wave::sync();
        uint32_t first[K], o[K];
        float high[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = k * 64 + lane < count;
            first[k] = in ? q->first[k * 64 + lane] : 0;
            high[k] = in ? q->high[k * 64 + lane] : 0.f;
            const uint32_t b = bits_of(high[k] + 0.f);
            o[k] = in ? b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u) : 0;  // ordered; 0 is below all
        }
        uint32_t x = 0;  // the largest number that `top` of them reach, bit by bit
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t y = x | (1u << bit);
            int n = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) n += __builtin_popcountll(Wave::ballot(o[k] >= y));
            if (n >= top) x = y;
        }
        Wave::sync();
        int kept = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = o[k] != 0 && o[k] >= x;
            const uint64_t m = Wave::ballot(in);
            if (in) {
                const int at = kept + __builtin_popcountll(m & ((1ull << lane) - 1));
                q->first[at] = first[k];
                q->high[at] = high[k];
            }
            kept += __builtin_popcountll(m);
        }
        count = kept;
        if (x) {
            bound = float_of(x ^ ((x >> 31) ? 0x80000000u : 0xffffffffu));
            thr = bound < __builtin_inff() ? fmaxf(thr, next_above(bound)) : __builtin_nanf("");
        }
        Wave::sync();
    }
};

}  // namespace
}  // namespace msscan
