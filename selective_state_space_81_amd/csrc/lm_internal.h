// lm_internal.h -- launch interface between the C ABI of the language-model
// operators beside the scan (lm_api.cpp) and their kernels (gated_scan.hip,
// embed.hip, logprob.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace msscan {

// Workgroups of 256 threads that one launch may have: a grid's threads are
// counted in 32 bits.
constexpr int64_t kMaxGroups = (1 << 24) - 1;

// ---- gated linear recurrence (gated_scan.hip) --------------------------------
// Saved states: h before every kGatedBlock-th step, [batch][ceil(L/kGatedBlock)][Dn].
constexpr int kGatedBlock = 16;

struct GatedArgs {
    const void* x;  // x, r, i, z: rows `ld` values apart
    const void* r;
    const void* i;
    const void* z;         // or null
    const float* lam;      // [Dn]
    const uint8_t* reset;  // [batch][L] or null
    const float* h0;       // [batch][Dn] or null
    void* y;
    float* h_last;  // [batch][Dn] or null
    float* states;  // forward: written (or null); backward: read
    // backward
    const void* dy;
    const float* dh_last;  // or null
    void* dx;
    void* dr;
    void* di;
    void* dz;
    float* dlam;
    float* dh0;   // or null
    float* part;  // workspace: partial sums of dlam, [batch][blocks][Dn]
    // workspace of blocks on workgroups of their own
    uint32_t* ticket;  // [chains], spaced: blocks of each handed out
    uint64_t* word;    // [chains][blocks][channels of a chain]: messages of the blocks
    int64_t blocks;    // blocks of a chain
    uint32_t chains;   // channel tiles of all batch rows
    float sharp;
    int64_t L;
    int64_t nstates;  // ceil(L / kGatedBlock)
    int64_t ld;
    int batch;
    int Dn;
};

int64_t gated_workgroups(int batch, int64_t L, int Dn, bool bf16);  // of the larger of both passes
size_t gated_fwd_ws(int batch, int64_t L, int Dn, bool bf16);  // bytes
size_t gated_bwd_ws(int batch, int64_t L, int Dn, bool bf16);
hipError_t launch_gated_fwd(GatedArgs a, bool bf16, void* workspace, hipStream_t s);
hipError_t launch_gated_bwd(GatedArgs a, bool bf16, void* workspace, hipStream_t s);
int64_t gated_step_workgroups(const GatedArgs& a);
// One step: a.h_last is the state [batch][Dn], updated in place; L is 1.
hipError_t launch_gated_step(const GatedArgs& a, bool bf16, hipStream_t s);

// ---- embedding (embed.hip) ----------------------------------------------------
constexpr int kDigitBits = 9;   // sort digit: two passes up to 2^18 tokens
constexpr int kMaxTiles = 256;  // sort workgroups
constexpr int kFew = 256;       // entries that are not sorted
constexpr int kSmall = 6144;    // entries one workgroup sorts

struct EmbedArgs {
    const void* ids;     // [n], int32 or int64
    const void* weight;  // [rows][D]
    void* out;           // [n][D]
    const void* dy;      // [n][D]
    void* dweight;       // [rows][D]
    float* part;         // [chunks][2][D]: pieces of runs that cross chunks
    float scale;
    int wide;  // ids are int64
    int64_t n;
    int64_t rows;
    int64_t padding;  // token without a gradient, or -1
    int D;
    // plan of the gradient
    int64_t tile;  // entries a sort workgroup takes
    int tiles;
    int passes;
    int bits;       // of a pass's digit
    int few;        // no sort
    int small;      // one workgroup sorts
    int lanes;      // threads that share a piece of the sums
    int64_t chunk;  // sorted entries in a piece
    int64_t chunks;  // without a sort, the entries
    int64_t zeros;  // pieces that write rows of tokens that do not occur
    int64_t sums;   // without a sort: workgroups of the sums, before those of zeros
};
struct SortPass {
    const uint32_t* key_in;
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    uint32_t* hist;  // [tiles][1 << kDigitBits]
    int shift;
    uint32_t mask;
    int first;  // keys come from the ids, positions are the entries' own
};
struct EmbedWs {
    size_t hist, key[2], pos[2], part, total;
};
int embed_vec(int D, bool bf16);
void embed_plan(EmbedArgs& a, bool bf16);  // from n, rows, D
EmbedWs embed_ws(const EmbedArgs& a);
int64_t embed_fwd_workgroups(const EmbedArgs& a, bool bf16);
int64_t embed_sum_workgroups(const EmbedArgs& a, bool bf16, bool gbf16);
hipError_t launch_embed_fwd(const EmbedArgs& a, bool bf16, hipStream_t s);
hipError_t launch_embed_bwd(EmbedArgs a, bool bf16, bool gbf16, void* workspace, hipStream_t s);

// ---- token log probabilities (logprob.hip) --------------------------------------
constexpr int kMaxTop = 64;  // alternatives a row can ask for: one a lane

struct LogprobArgs {
    const void* logits;  // [rows][ld], the first V of each row
    const void* targets;  // [rows], int32 or int64, or null
    float* logprob;       // [rows] or null
    float* entropy;       // [rows] or null
    float* lse;           // [rows] or null
    float* stats;         // [rows][2] or null: largest logit, ln of the sum beside it
    float* top_logprob;   // [rows][top]
    int32_t* top_id;      // [rows][top]
    // backward
    const float* dlogprob;  // [rows] or null
    const float* dentropy;  // [rows] or null
    void* dlogits;          // [rows][ldd]
    // workspace: per (row, split) partial sums and sorted keys
    float* part;     // [rows][splits][4]
    uint64_t* list;  // [rows][splits][top]
    float scale;
    int wide;
    int64_t rows;
    int64_t V;
    int64_t ld;
    int64_t ldd;
    int top;
    int splits;    // workgroups of a row
    int waves;     // of a workgroup, 4 or 16
    uint32_t per;  // vectors each of them takes
};
struct LogprobWs {
    size_t part, list, total;
};
void logprob_plan(LogprobArgs& a, bool bf16);  // splits, from rows and V
LogprobWs logprob_ws(const LogprobArgs& a);
hipError_t launch_logprob_fwd(LogprobArgs a, bool bf16, void* workspace, hipStream_t s);
int64_t logprob_bwd_workgroups(const LogprobArgs& a, bool bf16);
hipError_t launch_logprob_bwd(const LogprobArgs& a, bool bf16, hipStream_t s);

}  // namespace msscan
