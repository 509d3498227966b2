// lm_api.cpp -- the C ABI of the language-model operators beside the scan:
// the gated linear recurrence, the embedding and the token log probabilities.
// Argument validation and dispatch; the contract is in include/msscan.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/msscan.h"
#include "lm_internal.h"
#include "msscan_internal.h"

namespace {

using namespace msscan;

ms_status fail(ms_status s, const char* fmt, ...) {
    char text[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return report(s, text);
}

constexpr int64_t kMax31 = 0x7fffffffLL;
constexpr int64_t kMaxRowBytes = (1 << 24) - 1;  // of the gated scan: offsets are 24-bit products

ms_status check_aligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u)
            return fail(MS_ERR_ALIGN, "pointer %p is not 16-byte aligned", p);
    return MS_OK;
}

// What is read element by element, or in vectors that assume no more.
ms_status check_element_aligned(size_t size, std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1))
            return fail(MS_ERR_ALIGN, "pointer %p is not aligned to its element", p);
    return MS_OK;
}

size_t io_size(int32_t io) { return io == MS_BF16 ? 2 : 4; }

ms_status check_io(int32_t io, const char* name = "io") {
    if (io != MS_F32 && io != MS_BF16)
        return fail(MS_ERR_DTYPE, "%s=%d is not MS_F32 (0) or MS_BF16 (1)", name, io);
    return MS_OK;
}

ms_status check_id_bits(int32_t bits) {
    if (bits != 32 && bits != 64) return fail(MS_ERR_DTYPE, "id_bits=%d is not 32 or 64", bits);
    return MS_OK;
}

ms_status check_workspace(size_t need, const void* workspace, size_t given) {
    if (need && (!workspace || given < need))
        return fail(MS_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? given : (size_t)0);
    return MS_OK;
}

ms_status launched(hipError_t e) {
    return e == hipSuccess ? MS_OK : fail(MS_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

// ---- gated linear recurrence ---------------------------------------------------

ms_status check_gated_sizes(int32_t batch, int64_t seqlen, int32_t d_inner, int32_t io) {
    if (batch < 1) return fail(MS_ERR_SHAPE, "batch=%d must be >= 1", batch);
    if (seqlen < 1 || seqlen > kMax31)
        return fail(MS_ERR_SHAPE, "seqlen=%lld must be in [1, 2^31-1]", (long long)seqlen);
    if (d_inner < 1) return fail(MS_ERR_SHAPE, "d_inner=%d must be >= 1", d_inner);
    if ((double)batch * (double)seqlen * (double)d_inner > 0x1p56)
        return fail(MS_ERR_SHAPE, "batch x seqlen x d_inner exceeds 2^56");
    return check_io(io);
}

ms_status check_gated(int32_t batch, int64_t seqlen, int32_t d_inner, int32_t io) {
    ms_status st = check_gated_sizes(batch, seqlen, d_inner, io);
    if (st != MS_OK) return st;
    if ((d_inner + 63) / 64 > 65535 || batch > 65535)
        return fail(MS_ERR_UNSUPPORTED, "d_inner/64 and batch must be <= 65535");
    if (gated_workgroups(batch, seqlen, d_inner, io == MS_BF16) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "batch x seqlen x d_inner needs more than 2^24-1 workgroups");
    return MS_OK;
}

ms_status check_sharpness(float c) {
    if (!(c > 0.f) || !std::isfinite(c))
        return fail(MS_ERR_SHAPE, "sharpness=%g must be > 0 and finite", (double)c);
    return MS_OK;
}

// Rows of x, r, i and z, `most` bytes long at the most, and their alignment.
ms_status check_rows(int32_t d_inner, int64_t ld, int32_t io, int64_t most,
                     std::initializer_list<const void*> ptrs) {
    if (ld < d_inner) return fail(MS_ERR_SHAPE, "ld=%lld is below d_inner", (long long)ld);
    if (ld > most / (int64_t)io_size(io))
        return fail(MS_ERR_UNSUPPORTED, "rows of ld=%lld values are too long", (long long)ld);
    return ld == d_inner ? check_aligned(ptrs) : check_element_aligned(io_size(io), ptrs);
}

int64_t state_rows(int64_t seqlen) { return (seqlen + kGatedBlock - 1) / kGatedBlock; }

// ---- embedding -------------------------------------------------------------------

ms_status check_embed(int64_t n, int64_t rows, int32_t dim, int32_t io) {
    if (n < 0 || n > kMax31)
        return fail(MS_ERR_SHAPE, "n=%lld must be in [0, 2^31-1]", (long long)n);
    if (rows < 1 || rows > kMax31)
        return fail(MS_ERR_SHAPE, "rows=%lld must be in [1, 2^31-1]", (long long)rows);
    if (dim < 1 || dim > (1 << 24)) return fail(MS_ERR_SHAPE, "dim=%d must be in [1, 2^24]", dim);
    return check_io(io);
}

// ---- token log probabilities -------------------------------------------------------

ms_status check_logprobs(int64_t rows, int64_t vocab, int32_t top, int32_t io) {
    if (rows < 0 || rows > kMax31)
        return fail(MS_ERR_SHAPE, "rows=%lld must be in [0, 2^31-1]", (long long)rows);
    if (vocab < 1 || vocab > kMax31)
        return fail(MS_ERR_SHAPE, "vocab=%lld must be in [1, 2^31-1]", (long long)vocab);
    if (rows > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "rows=%lld must be below 2^24", (long long)rows);
    if (top < 0 || top > kMaxTop || top > vocab)
        return fail(MS_ERR_SHAPE, "top=%d must be in [0, %d] and at most vocab", top, kMaxTop);
    return check_io(io);
}

ms_status check_scale(float scale, bool positive) {
    if (!std::isfinite(scale) || (positive && !(scale > 0.f)))
        return fail(MS_ERR_SHAPE, "scale=%g must be finite%s", (double)scale,
                    positive ? " and > 0" : "");
    return MS_OK;
}

}  // namespace

extern "C" {

size_t ms_gated_scan_workspace_bytes(int32_t batch, int64_t seqlen, int32_t d_inner, int32_t io) {
    if (check_gated(batch, seqlen, d_inner, io) != MS_OK) return (size_t)-1;
    return gated_fwd_ws(batch, seqlen, d_inner, io == MS_BF16);
}

size_t ms_gated_scan_states_bytes(int32_t batch, int64_t seqlen, int32_t d_inner) {
    if (check_gated(batch, seqlen, d_inner, MS_F32) != MS_OK) return (size_t)-1;
    return (size_t)batch * (size_t)state_rows(seqlen) * (size_t)d_inner * sizeof(float);
}

ms_status ms_gated_scan_fwd(const void* x, const void* r, const void* i, const float* lam,
                            float sharpness, const void* z, const uint8_t* reset, void* y,
                            const float* h0, float* h_last, float* states, int32_t batch,
                            int64_t seqlen, int32_t d_inner, int64_t ld, int32_t io,
                            void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    ms_status st = check_gated(batch, seqlen, d_inner, io);
    if (st != MS_OK) return st;
    if ((st = check_sharpness(sharpness)) != MS_OK) return st;
    if (!x || !r || !i || !lam || !y) return fail(MS_ERR_NULL, "x, r, i, lam and y are required");
    if ((st = check_rows(d_inner, ld, io, kMaxRowBytes, {x, r, i, z})) != MS_OK) return st;
    if ((st = check_aligned({y, h0, h_last, states, workspace})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {lam})) != MS_OK) return st;
    if ((st = check_workspace(ms_gated_scan_workspace_bytes(batch, seqlen, d_inner, io), workspace,
                              workspace_bytes)) != MS_OK)
        return st;
    GatedArgs a{};
    a.x = x; a.r = r; a.i = i; a.z = z; a.lam = lam; a.reset = reset; a.h0 = h0; a.y = y;
    a.h_last = h_last; a.states = states; a.sharp = sharpness; a.L = seqlen;
    a.nstates = state_rows(seqlen); a.batch = batch; a.Dn = d_inner; a.ld = ld;
    prof_call();
    return launched(launch_gated_fwd(a, io == MS_BF16, workspace, static_cast<hipStream_t>(stream)));
}

size_t ms_gated_scan_bwd_workspace_bytes(int32_t batch, int64_t seqlen, int32_t d_inner,
                                         int32_t io) {
    if (check_gated(batch, seqlen, d_inner, io) != MS_OK) return (size_t)-1;
    return gated_bwd_ws(batch, seqlen, d_inner, io == MS_BF16);
}

ms_status ms_gated_scan_bwd(const void* x, const void* r, const void* i, const float* lam,
                            float sharpness, const void* z, const uint8_t* reset,
                            const float* states, const void* dy, const float* dh_last, void* dx,
                            void* dr, void* di, void* dz, float* dlam, float* dh0, int32_t batch,
                            int64_t seqlen, int32_t d_inner, int64_t ld, int32_t io,
                            void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    ms_status st = check_gated(batch, seqlen, d_inner, io);
    if (st != MS_OK) return st;
    if ((st = check_sharpness(sharpness)) != MS_OK) return st;
    if (!x || !r || !i || !lam || !states || !dy || !dx || !dr || !di || !dlam)
        return fail(MS_ERR_NULL, "x, r, i, lam, states, dy, dx, dr, di and dlam are required");
    if (z && !dz) return fail(MS_ERR_NULL, "dz is required when z is given");
    if ((st = check_rows(d_inner, ld, io, kMaxRowBytes, {x, r, i, z})) != MS_OK) return st;
    if ((st = check_aligned({states, dx, dr, di, dz, dlam, dh0, workspace})) != MS_OK) return st;
    if ((st = check_element_aligned(io_size(io), {dy})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {lam, dh_last})) != MS_OK) return st;
    if ((st = check_workspace(ms_gated_scan_bwd_workspace_bytes(batch, seqlen, d_inner, io),
                              workspace, workspace_bytes)) != MS_OK)
        return st;
    GatedArgs a{};
    a.x = x; a.r = r; a.i = i; a.z = z; a.lam = lam; a.reset = reset; a.dy = dy;
    a.states = const_cast<float*>(states);  // only read
    a.dh_last = dh_last; a.dx = dx; a.dr = dr; a.di = di; a.dz = dz; a.dlam = dlam; a.dh0 = dh0;
    a.sharp = sharpness; a.L = seqlen;
    a.nstates = state_rows(seqlen); a.batch = batch; a.Dn = d_inner; a.ld = ld;
    prof_call();
    return launched(launch_gated_bwd(a, io == MS_BF16, workspace, static_cast<hipStream_t>(stream)));
}

ms_status ms_gated_step(float* h, const void* x_t, const void* r_t, const void* i_t,
                        const float* lam, float sharpness, const void* z_t, void* y_t,
                        int32_t batch, int32_t d_inner, int64_t ld, int32_t io, void* stream) {
    clear_error();
    ms_status st = check_gated_sizes(batch, 1, d_inner, io);
    if (st != MS_OK) return st;
    if ((st = check_sharpness(sharpness)) != MS_OK) return st;
    if (!h || !x_t || !r_t || !i_t || !lam || !y_t)
        return fail(MS_ERR_NULL, "h, x_t, r_t, i_t, lam and y_t are required");
    if ((st = check_rows(d_inner, ld, io, (int64_t)1 << 40, {x_t, r_t, i_t, z_t})) != MS_OK)
        return st;
    if ((st = check_aligned({h, y_t})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {lam})) != MS_OK) return st;
    GatedArgs a{};
    a.x = x_t; a.r = r_t; a.i = i_t; a.z = z_t; a.lam = lam; a.h_last = h; a.y = y_t;
    a.sharp = sharpness; a.L = 1; a.batch = batch; a.Dn = d_inner; a.ld = ld;
    if (gated_step_workgroups(a) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "batch x d_inner needs more than 2^24-1 workgroups");
    prof_call();
    return launched(launch_gated_step(a, io == MS_BF16, static_cast<hipStream_t>(stream)));
}

ms_status ms_embed_fwd(const void* ids, int32_t id_bits, const void* weight, float scale,
                       void* out, int64_t n, int64_t rows, int32_t dim, int32_t io,
                       void* stream) {
    clear_error();
    ms_status st = check_embed(n, rows, dim, io);
    if (st != MS_OK) return st;
    if ((st = check_id_bits(id_bits)) != MS_OK) return st;
    if ((st = check_scale(scale, false)) != MS_OK) return st;
    if (n == 0) return MS_OK;
    if (!ids || !weight || !out) return fail(MS_ERR_NULL, "ids, weight and out are required");
    if ((st = check_aligned({weight, out})) != MS_OK) return st;
    if ((st = check_element_aligned(id_bits / 8, {ids})) != MS_OK) return st;
    EmbedArgs a{};
    a.ids = ids; a.wide = id_bits == 64; a.weight = weight; a.scale = scale; a.out = out; a.n = n;
    a.rows = rows; a.D = dim;
    if (embed_fwd_workgroups(a, io == MS_BF16) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "n x dim needs more than 2^24-1 workgroups");
    prof_call();
    return launched(launch_embed_fwd(a, io == MS_BF16, static_cast<hipStream_t>(stream)));
}

size_t ms_embed_bwd_workspace_bytes(int64_t n, int64_t rows, int32_t dim, int32_t io) {
    if (check_embed(n, rows, dim, io) != MS_OK) return (size_t)-1;
    EmbedArgs a{};
    a.n = n; a.rows = rows; a.D = dim;
    embed_plan(a, io == MS_BF16);
    return embed_ws(a).total;
}

ms_status ms_embed_bwd(const void* ids, int32_t id_bits, const void* dy, float scale,
                       int64_t padding, void* dweight, int32_t grad_dtype, int64_t n,
                       int64_t rows, int32_t dim, int32_t io, void* workspace,
                       size_t workspace_bytes, void* stream) {
    clear_error();
    ms_status st = check_embed(n, rows, dim, io);
    if (st != MS_OK) return st;
    if ((st = check_io(grad_dtype, "grad_dtype")) != MS_OK) return st;
    if ((st = check_id_bits(id_bits)) != MS_OK) return st;
    if ((st = check_scale(scale, false)) != MS_OK) return st;
    if (!dweight || (n && (!ids || !dy)))
        return fail(MS_ERR_NULL, "ids, dy and dweight are required");
    if ((st = check_aligned({dweight, workspace})) != MS_OK) return st;
    if ((st = check_element_aligned(id_bits / 8, {ids})) != MS_OK) return st;
    if ((st = check_element_aligned(io_size(io), {dy})) != MS_OK) return st;
    EmbedArgs a{};
    a.ids = ids; a.wide = id_bits == 64; a.dy = dy; a.scale = scale; a.padding = padding;
    a.dweight = dweight; a.n = n; a.rows = rows; a.D = dim;
    embed_plan(a, io == MS_BF16);
    if ((st = check_workspace(embed_ws(a).total, workspace, workspace_bytes)) != MS_OK) return st;
    if (embed_sum_workgroups(a, io == MS_BF16, grad_dtype == MS_BF16) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "n, rows and dim need more than 2^24-1 workgroups");
    prof_call();
    return launched(launch_embed_bwd(a, io == MS_BF16, grad_dtype == MS_BF16, workspace,
                                     static_cast<hipStream_t>(stream)));
}

size_t ms_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t top, int32_t io) {
    if (check_logprobs(rows, vocab, top, io) != MS_OK) return (size_t)-1;
    LogprobArgs a{};
    a.rows = rows; a.V = vocab; a.top = top;
    logprob_plan(a, io == MS_BF16);
    return logprob_ws(a).total;
}

ms_status ms_token_logprobs_fwd(const void* logits, int64_t ld, const void* targets,
                                int32_t id_bits, float scale, float* logprob, float* entropy,
                                float* lse, float* stats, int32_t top, float* top_logprob,
                                int32_t* top_id, int64_t rows, int64_t vocab, int32_t io, void* workspace,
                                size_t workspace_bytes, void* stream) {
    clear_error();
    ms_status st = check_logprobs(rows, vocab, top, io);
    if (st != MS_OK) return st;
    if (ld < vocab) return fail(MS_ERR_SHAPE, "ld=%lld is below vocab", (long long)ld);
    if ((st = check_id_bits(id_bits)) != MS_OK) return st;
    if ((st = check_scale(scale, true)) != MS_OK) return st;
    if (rows == 0) return MS_OK;
    if (!logits || (logprob && !targets) || (top && (!top_logprob || !top_id)))
        return fail(MS_ERR_NULL, "logits are required, targets with logprob, and top_logprob and "
                                 "top_id with top");
    if ((st = check_aligned({logits, logprob, entropy, lse, stats, top_logprob, top_id, workspace})) !=
        MS_OK)
        return st;
    if ((st = check_element_aligned(id_bits / 8, {targets})) != MS_OK) return st;
    LogprobArgs a{};
    a.logits = logits; a.targets = targets; a.wide = id_bits == 64; a.logprob = logprob;
    a.entropy = entropy; a.lse = lse; a.stats = stats; a.top = top; a.top_logprob = top_logprob; a.top_id = top_id;
    a.scale = scale; a.rows = rows; a.V = vocab; a.ld = ld;
    logprob_plan(a, io == MS_BF16);
    if ((st = check_workspace(logprob_ws(a).total, workspace, workspace_bytes)) != MS_OK) return st;
    prof_call();
    return launched(
        launch_logprob_fwd(a, io == MS_BF16, workspace, static_cast<hipStream_t>(stream)));
}

ms_status ms_token_logprobs_bwd(const void* logits, int64_t ld, const void* targets,
                                int32_t id_bits, float scale, const float* stats,
                                const float* entropy, const float* dlogprob,
                                const float* dentropy, void* dlogits, int64_t ldd, int64_t rows,
                                int64_t vocab, int32_t io, void* stream) {
    clear_error();
    ms_status st = check_logprobs(rows, vocab, 0, io);
    if (st != MS_OK) return st;
    if (ld < vocab || ldd < vocab)
        return fail(MS_ERR_SHAPE, "ld=%lld or ldd=%lld is below vocab", (long long)ld,
                    (long long)ldd);
    if ((st = check_id_bits(id_bits)) != MS_OK) return st;
    if ((st = check_scale(scale, true)) != MS_OK) return st;
    if (rows == 0) return MS_OK;
    if (!logits || !stats || !dlogits || (dlogprob && !targets) || (dentropy && !entropy))
        return fail(MS_ERR_NULL, "logits, stats and dlogits are required, targets with dlogprob, and "
                                 "entropy with dentropy");
    if (dlogits == logits && ld != ldd)
        return fail(MS_ERR_SHAPE, "dlogits over logits needs ldd == ld");
    if ((st = check_aligned({logits, dlogits})) != MS_OK) return st;
    if ((st = check_element_aligned(id_bits / 8, {targets})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {stats, entropy, dlogprob, dentropy})) != MS_OK) return st;
    LogprobArgs a{};
    a.logits = logits; a.targets = targets; a.wide = id_bits == 64;
    a.stats = const_cast<float*>(stats);      // only read
    a.entropy = const_cast<float*>(entropy);  // only read
    a.dlogprob = dlogprob; a.dentropy = dentropy; a.dlogits = dlogits; a.scale = scale;
    a.rows = rows; a.V = vocab; a.ld = ld; a.ldd = ldd;
    if (logprob_bwd_workgroups(a, io == MS_BF16) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "rows x vocab needs more than 2^24-1 workgroups");
    prof_call();
    return launched(launch_logprob_bwd(a, io == MS_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
