// lm_internal.h -- launch interface between the C ABI of the language-model
// operators beside the scan (lm_api.cpp, attn_api.cpp) and their kernels
// (gated_scan.hip, embed.hip, logprob.hip; linear_attn*.hip, group_norm.hip,
// verify.hip).  Not part of the public ABI.
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

// ---- linear attention (linear_attn.hip, linear_attn_bwd.hip) ----------------------
constexpr int kAttnBlockBf16 = 64;  // tokens of a block
constexpr int kAttnBlockF32 = 32;
constexpr int kMaxHeadDim = 128;  // of dk and dv
constexpr int kStepTokens = 64;   // most tokens of a step

struct AttnArgs {
    const void* q;  // [batch][L] rows ldq apart, of Hk heads of dk
    const void* k;
    const void* v;         // of H heads of dv
    const float* g;        // [batch][L][H], or [H] (fixed)
    const uint8_t* reset;  // [batch][L] or null
    const float* h0;       // [batch][H][dk][dv] or null
    void* o;               // [batch][L][H][dv]
    float* h_last;         // [batch][H][dk][dv] or null
    float* states;         // [batch][blocks][H][DKs][DVs]; forward: written, or null
    // backward
    const void* dO;
    const float* dh_last;
    void* dq;
    void* dk_out;
    void* dv_out;
    float* dg;   // [batch][L][H], or [H] (fixed)
    float* dh0;  // or null
    // step
    float* h;
    const int32_t* counts;  // [batch] or null
    int update;
    // workspace
    float* seg;     // [batch][nseg][H][dk][dv]: states at the ends, then the starts, of segments
    float* seg_f;   // [batch][nseg][H]: decay of a segment, -1 where a document starts in it
    float* grads;   // [batch][blocks][H][DKs][DVs]: gradients of the states at the blocks' ends
    float* part;    // [batch][blocks][H]: sums of a fixed decay's gradient
    int64_t ldq, ldk, ldv;
    int64_t L;
    int64_t blocks;
    int64_t per;  // blocks of a segment
    float scale;
    int nseg;
    int fixed;
    int batch, H, Hk, dk, dv;
    int DKs, DVs;  // dk and dv in whole tiles of 16
    int tiles;     // tiles of 64 columns of dv
};
struct AttnWs {
    size_t seg, seg_f, grads, part, total;
};
void attn_plan(AttnArgs& a, bool bf16);
AttnWs attn_ws(const AttnArgs& a, bool backward);
int64_t attn_workgroups(const AttnArgs& a, bool backward);  // the most of a launch, as of 256 threads
hipError_t launch_attn_fwd(AttnArgs a, bool bf16, void* workspace, hipStream_t s);
hipError_t launch_attn_bwd(AttnArgs a, bool bf16, void* workspace, hipStream_t s);
// The walk of the states alone, forward in time (k, v) or backward (q, dO).  Not
// full: sums of all segments but the last, to a.seg and a.seg_f.  Full (backward
// only): from the segments' starts, each block's to a.grads and the last to a.dh0.
hipError_t launch_attn_walk(const AttnArgs& a, bool bf16, bool reverse, bool full, hipStream_t s);
hipError_t launch_attn_carry(const AttnArgs& a, const float* first, hipStream_t s);
int64_t attn_step_workgroups(const AttnArgs& a);
hipError_t launch_attn_step(const AttnArgs& a, bool bf16, hipStream_t s);

// ---- group norm of each row's channels (group_norm.hip) ------------------------------
constexpr int kMaxNormGroup = 8192;  // channels of a group

struct NormArgs {
    const void* x;  // [rows], ldx apart, of groups * size
    const void* z;  // [rows], ldz apart, or null
    const float* weight;  // [groups * size] or null
    const float* bias;    // or null
    void* y;              // [rows][groups * size]
    // backward
    const void* dy;
    void* dx;
    void* dz;
    float* dweight;  // or null
    float* dbias;    // or null
    float* part;     // [strips][2][groups * size]: sums of dweight and dbias
    int64_t ldx, ldz;
    int64_t rows;
    float eps;
    int groups, size;
    int center, gate_first;
    // plan
    int lanes;      // that share a group: a power of two, or 256 (a workgroup)
    int vecs;       // vectors of a lane
    int columns;    // workgroups side by side for a row's groups
    int64_t strips;  // workgroups one above the other
};
void norm_plan(NormArgs& a, bool bf16, bool backward);
size_t norm_bwd_ws(const NormArgs& a);
int64_t norm_workgroups(const NormArgs& a);
hipError_t launch_norm_fwd(const NormArgs& a, bool bf16, hipStream_t s);
hipError_t launch_norm_bwd(NormArgs a, bool bf16, void* workspace, hipStream_t s);

// ---- verification of drafted tokens (verify.hip) --------------------------------------
constexpr int kMaxDrafts = 64;

struct VerifyArgs {
    const void* logits;  // [batch][drafts + 1] rows ld apart
    const void* draft_logits;  // [batch][drafts] rows ldd apart, or null
    const void* tokens_in;     // [batch][drafts], int32 or int64
    const float* uniforms;     // [batch][drafts + 1]
    int32_t* tokens;           // [batch][drafts + 1]
    int32_t* count;            // [batch]
    float* logprob;            // [batch][drafts + 1]
    double* part;  // [rows][splits][2]: largest exponent, sum beside it
    double* mass;  // [batch][pieces][2]: of what is left, and of the target's
    uint32_t* done;  // [batch]: pieces whose mass is there
    int64_t ld, ldd;
    int64_t V;
    float scale;
    int wide;
    int batch, drafts;
    // plan
    int64_t rows;    // of both, the target's first
    int splits;      // workgroups of a row
    int64_t per;     // values each of them takes
    int pieces;      // of a row that is drawn from
    int piece;       // values of one
};
struct VerifyWs {
    size_t part, mass, done, total;
};
void verify_plan(VerifyArgs& a, bool bf16, bool drafted);
VerifyWs verify_ws(const VerifyArgs& a);
int64_t verify_workgroups(const VerifyArgs& a);
hipError_t launch_verify(VerifyArgs a, bool bf16, void* workspace, hipStream_t s);

}  // namespace msscan
