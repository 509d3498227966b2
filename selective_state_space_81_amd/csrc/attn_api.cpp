// attn_api.cpp -- the C ABI of the linear attention, the group norm and the
// verification of drafted tokens.  Argument validation and dispatch; the
// contract is in include/msscan.h.
#include "lm_checks.h"
#include "lm_internal.h"

namespace {

using namespace msscan;

// ---- linear attention ------------------------------------------------------------

ms_status check_attn(int32_t batch, int64_t seqlen, int32_t heads, int32_t kheads, int32_t dk,
                     int32_t dv, int32_t io) {
    if (batch < 1) return fail(MS_ERR_SHAPE, "batch=%d must be >= 1", batch);
    if (seqlen < 1 || seqlen > kMax31)
        return fail(MS_ERR_SHAPE, "seqlen=%lld must be in [1, 2^31-1]", (long long)seqlen);
    if (heads < 1) return fail(MS_ERR_SHAPE, "heads=%d must be >= 1", heads);
    if (kheads < 1 || heads % kheads)
        return fail(MS_ERR_SHAPE, "kheads=%d must divide heads=%d", kheads, heads);
    if (dk < 1) return fail(MS_ERR_SHAPE, "dk=%d must be >= 1", dk);
    if (dv < 1) return fail(MS_ERR_SHAPE, "dv=%d must be >= 1", dv);
    if ((double)batch * (double)seqlen * (double)heads * 256.0 > 0x1p56)
        return fail(MS_ERR_SHAPE, "batch x seqlen x heads exceeds 2^48");
    if (dk > kMaxHeadDim || dv > kMaxHeadDim)
        return fail(MS_ERR_UNSUPPORTED, "dk=%d and dv=%d must be <= %d", dk, dv, kMaxHeadDim);
    return check_io(io);
}

AttnArgs attn_args(int32_t batch, int64_t seqlen, int32_t heads, int32_t kheads, int32_t dk,
                   int32_t dv) {
    AttnArgs a{};
    a.batch = batch; a.L = seqlen; a.H = heads; a.Hk = kheads; a.dk = dk; a.dv = dv;
    return a;
}

// Sizes, and that every launch of the pass has a grid: the plan of them in `a`.
ms_status plan_attn(AttnArgs& a, int32_t batch, int64_t seqlen, int32_t heads, int32_t kheads,
                    int32_t dk, int32_t dv, int32_t io, bool backward) {
    ms_status st = check_attn(batch, seqlen, heads, kheads, dk, dv, io);
    if (st != MS_OK) return st;
    a = attn_args(batch, seqlen, heads, kheads, dk, dv);
    if ((double)batch * heads * 2.0 > 0x1p30)
        return fail(MS_ERR_UNSUPPORTED, "batch x heads needs more than 2^24-1 workgroups");
    attn_plan(a, io == MS_BF16);
    if (attn_workgroups(a, backward) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "batch x seqlen x heads needs more than 2^24-1 workgroups");
    return MS_OK;
}

ms_status check_pitch(const char* name, int64_t ld, int64_t width) {
    if (ld < width)
        return fail(MS_ERR_SHAPE, "%s=%lld is below the row's %lld values", name, (long long)ld,
                    (long long)width);
    if (ld > ((int64_t)1 << 40)) return fail(MS_ERR_UNSUPPORTED, "%s is too long", name);
    return MS_OK;
}

// Rows of q, k and v: 32 bits hold a place in a block of them.
ms_status check_rows_of_heads(int64_t ldq, int64_t ldk, int64_t ldv, int64_t qk, int64_t v) {
    ms_status st;
    if ((st = check_pitch("ldq", ldq, qk)) != MS_OK) return st;
    if ((st = check_pitch("ldk", ldk, qk)) != MS_OK) return st;
    if ((st = check_pitch("ldv", ldv, v)) != MS_OK) return st;
    const int64_t most = (1 << 22) - 1;
    if (ldq > most || ldk > most || ldv > most)
        return fail(MS_ERR_UNSUPPORTED, "rows of 2^22 values or more are too long");
    return MS_OK;
}

ms_status check_norm(NormArgs& a, int64_t rows, int32_t groups, int32_t size, float eps, int32_t io,
                     bool backward) {
    if (rows < 0 || rows > kMax31)
        return fail(MS_ERR_SHAPE, "rows=%lld must be in [0, 2^31-1]", (long long)rows);
    if (groups < 1) return fail(MS_ERR_SHAPE, "groups=%d must be >= 1", groups);
    if (size < 1) return fail(MS_ERR_SHAPE, "size=%d must be >= 1", size);
    if (!(eps > 0.f) || !std::isfinite(eps))
        return fail(MS_ERR_SHAPE, "eps=%g must be > 0 and finite", (double)eps);
    ms_status st = check_io(io);
    if (st != MS_OK) return st;
    if (size > kMaxNormGroup)
        return fail(MS_ERR_UNSUPPORTED, "size=%d must be <= %d", size, kMaxNormGroup);
    if ((int64_t)groups * size > (1 << 24))
        return fail(MS_ERR_UNSUPPORTED, "groups x size must be <= 2^24");
    a.rows = rows; a.groups = groups; a.size = size; a.eps = eps;
    norm_plan(a, io == MS_BF16, backward);
    if (norm_workgroups(a) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "groups need more than 2^24-1 workgroups");
    return MS_OK;
}

ms_status check_verify(VerifyArgs& a, int32_t batch, int32_t drafts, int64_t vocab, int32_t drafted,
                       int32_t io) {
    if (batch < 0) return fail(MS_ERR_SHAPE, "batch=%d must be >= 0", batch);
    if (drafts < 0 || drafts > kMaxDrafts)
        return fail(MS_ERR_SHAPE, "drafts=%d must be in [0, %d]", drafts, kMaxDrafts);
    if (vocab < 1 || vocab > kMax31)
        return fail(MS_ERR_SHAPE, "vocab=%lld must be in [1, 2^31-1]", (long long)vocab);
    ms_status st = check_io(io);
    if (st != MS_OK) return st;
    a.batch = batch; a.drafts = drafts; a.V = vocab;
    if (batch == 0) return MS_OK;
    verify_plan(a, io == MS_BF16, drafted != 0);
    if (verify_workgroups(a) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "batch x vocab needs more than 2^24-1 workgroups");
    return MS_OK;
}

}  // namespace

extern "C" {

size_t ms_linear_attn_workspace_bytes(int32_t batch, int64_t seqlen, int32_t heads, int32_t kheads,
                                      int32_t dk, int32_t dv, int32_t io) {
    AttnArgs a;
    if (plan_attn(a, batch, seqlen, heads, kheads, dk, dv, io, false) != MS_OK) return (size_t)-1;
    return attn_ws(a, false).total;
}

size_t ms_linear_attn_states_bytes(int32_t batch, int64_t seqlen, int32_t heads, int32_t dk,
                                   int32_t dv, int32_t io) {
    AttnArgs a;  // of the backward with one head of keys, which needs the fewest workgroups
    if (plan_attn(a, batch, seqlen, heads, 1, dk, dv, io, true) != MS_OK) return (size_t)-1;
    return (size_t)batch * a.blocks * heads * a.DKs * a.DVs * sizeof(float);
}

ms_status ms_linear_attn_fwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, const float* g, int32_t fixed, float scale,
                             const uint8_t* reset, void* o, const float* h0, float* h_last,
                             float* states, int32_t batch, int64_t seqlen, int32_t heads,
                             int32_t kheads, int32_t dk, int32_t dv, int32_t io, void* workspace,
                             size_t workspace_bytes, void* stream) {
    clear_error();
    AttnArgs a;
    ms_status st = plan_attn(a, batch, seqlen, heads, kheads, dk, dv, io, false);
    if (st != MS_OK) return st;
    if ((st = check_scale(scale, false)) != MS_OK) return st;
    if (!q || !k || !v || !g || !o) return fail(MS_ERR_NULL, "q, k, v, g and o are required");
    if ((st = check_rows_of_heads(ldq, ldk, ldv, (int64_t)kheads * dk, (int64_t)heads * dv)) != MS_OK)
        return st;
    if ((st = check_aligned({o, h0, h_last, states, workspace})) != MS_OK) return st;
    if ((st = check_element_aligned(io_size(io), {q, k, v})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {g})) != MS_OK) return st;
    if ((st = check_workspace(attn_ws(a, false).total, workspace, workspace_bytes)) != MS_OK)
        return st;
    a.q = q; a.ldq = ldq; a.k = k; a.ldk = ldk; a.v = v; a.ldv = ldv; a.g = g; a.fixed = fixed;
    a.scale = scale; a.reset = reset; a.o = o; a.h0 = h0; a.h_last = h_last; a.states = states;
    prof_call();
    return launched(launch_attn_fwd(a, io == MS_BF16, workspace, static_cast<hipStream_t>(stream)));
}

size_t ms_linear_attn_bwd_workspace_bytes(int32_t batch, int64_t seqlen, int32_t heads,
                                          int32_t kheads, int32_t dk, int32_t dv, int32_t fixed,
                                          int32_t io) {
    AttnArgs a;
    if (plan_attn(a, batch, seqlen, heads, kheads, dk, dv, io, true) != MS_OK) return (size_t)-1;
    a.fixed = fixed;
    return attn_ws(a, true).total;
}

ms_status ms_linear_attn_bwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, const float* g, int32_t fixed, float scale,
                             const uint8_t* reset, const float* states, const void* d_o,
                             const float* dh_last, void* dq, void* d_k, void* d_v, float* dg,
                             float* dh0, int32_t batch, int64_t seqlen, int32_t heads,
                             int32_t kheads, int32_t dk, int32_t dv, int32_t io, void* workspace,
                             size_t workspace_bytes, void* stream) {
    clear_error();
    AttnArgs a;
    ms_status st = plan_attn(a, batch, seqlen, heads, kheads, dk, dv, io, true);
    if (st != MS_OK) return st;
    if ((st = check_scale(scale, false)) != MS_OK) return st;
    if (!q || !k || !v || !g || !states || !d_o || !dq || !d_k || !d_v || !dg)
        return fail(MS_ERR_NULL, "q, k, v, g, states, d_o, dq, d_k, d_v and dg are required");
    if ((st = check_rows_of_heads(ldq, ldk, ldv, (int64_t)kheads * dk, (int64_t)heads * dv)) != MS_OK)
        return st;
    if ((st = check_aligned({states, dq, d_k, d_v, dg, dh0, workspace})) != MS_OK) return st;
    if ((st = check_element_aligned(io_size(io), {q, k, v, d_o})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {g, dh_last})) != MS_OK) return st;
    a.fixed = fixed;
    if ((st = check_workspace(attn_ws(a, true).total, workspace, workspace_bytes)) != MS_OK)
        return st;
    a.q = q; a.ldq = ldq; a.k = k; a.ldk = ldk; a.v = v; a.ldv = ldv; a.g = g; a.scale = scale;
    a.reset = reset; a.states = const_cast<float*>(states);  // only read
    a.dO = d_o; a.dh_last = dh_last; a.dq = dq; a.dk_out = d_k; a.dv_out = d_v; a.dg = dg;
    a.dh0 = dh0;
    prof_call();
    return launched(launch_attn_bwd(a, io == MS_BF16, workspace, static_cast<hipStream_t>(stream)));
}

ms_status ms_linear_attn_step(float* h, const void* q, int64_t ldq, const void* k, int64_t ldk,
                              const void* v, int64_t ldv, const float* g, int32_t fixed,
                              float scale, const int32_t* counts, int32_t update, void* o,
                              int32_t batch, int32_t tokens, int32_t heads, int32_t kheads,
                              int32_t dk, int32_t dv, int32_t io, void* stream) {
    clear_error();
    ms_status st = check_attn(batch, tokens, heads, kheads, dk, dv, io);
    if (st != MS_OK) return st;
    if (tokens > kStepTokens)
        return fail(MS_ERR_UNSUPPORTED, "tokens=%d must be <= %d", tokens, kStepTokens);
    if ((st = check_scale(scale, false)) != MS_OK) return st;
    if (!h || !k || !v || !g || (q && !o))
        return fail(MS_ERR_NULL, "h, k, v and g are required, and o with q");
    if (!q && !update) return fail(MS_ERR_NULL, "q is required without update");
    if (q && (st = check_pitch("ldq", ldq, (int64_t)kheads * dk)) != MS_OK) return st;
    if ((st = check_pitch("ldk", ldk, (int64_t)kheads * dk)) != MS_OK) return st;
    if ((st = check_pitch("ldv", ldv, (int64_t)heads * dv)) != MS_OK) return st;
    if ((st = check_aligned({h, q ? o : nullptr})) != MS_OK) return st;
    if ((st = check_element_aligned(io_size(io), {q, k, v})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {g, counts})) != MS_OK) return st;
    AttnArgs a = attn_args(batch, tokens, heads, kheads, dk, dv);
    a.tiles = (dv + 63) / 64;
    if (attn_step_workgroups(a) > kMaxGroups)
        return fail(MS_ERR_UNSUPPORTED, "batch x heads needs more than 2^24-1 workgroups");
    a.h = h; a.q = q; a.ldq = ldq; a.k = k; a.ldk = ldk; a.v = v; a.ldv = ldv; a.g = g;
    a.fixed = fixed; a.scale = scale; a.counts = counts; a.update = update; a.o = o;
    prof_call();
    return launched(launch_attn_step(a, io == MS_BF16, static_cast<hipStream_t>(stream)));
}

ms_status ms_group_norm_fwd(const void* x, int64_t ldx, const float* weight, const float* bias,
                            const void* z, int64_t ldz, int32_t center, int32_t gate_first,
                            float eps, void* y, int64_t rows, int32_t groups, int32_t size,
                            int32_t io, void* stream) {
    clear_error();
    NormArgs a{};
    ms_status st = check_norm(a, rows, groups, size, eps, io, false);
    if (st != MS_OK) return st;
    const int64_t width = (int64_t)groups * size;
    if ((st = check_pitch("ldx", ldx, width)) != MS_OK) return st;
    if (z && (st = check_pitch("ldz", ldz, width)) != MS_OK) return st;
    if (gate_first && !z) return fail(MS_ERR_NULL, "z is required with gate_first");
    if (rows == 0) return MS_OK;
    if (!x || !y) return fail(MS_ERR_NULL, "x and y are required");
    if ((st = check_aligned({y})) != MS_OK) return st;
    if ((st = check_element_aligned(io_size(io), {x, z})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {weight, bias})) != MS_OK) return st;
    a.x = x; a.ldx = ldx; a.weight = weight; a.bias = bias; a.z = z; a.ldz = ldz;
    a.center = center; a.gate_first = gate_first; a.y = y;
    prof_call();
    return launched(launch_norm_fwd(a, io == MS_BF16, static_cast<hipStream_t>(stream)));
}

size_t ms_group_norm_bwd_workspace_bytes(int64_t rows, int32_t groups, int32_t size, int32_t io) {
    NormArgs a{};
    if (check_norm(a, rows, groups, size, 1.f, io, true) != MS_OK) return (size_t)-1;
    return norm_bwd_ws(a);
}

ms_status ms_group_norm_bwd(const void* x, int64_t ldx, const float* weight, const float* bias,
                            const void* z, int64_t ldz, int32_t center, int32_t gate_first,
                            float eps, const void* dy, void* dx, void* dz, float* dweight,
                            float* dbias, int64_t rows, int32_t groups, int32_t size, int32_t io,
                            void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    NormArgs a{};
    ms_status st = check_norm(a, rows, groups, size, eps, io, true);
    if (st != MS_OK) return st;
    const int64_t width = (int64_t)groups * size;
    if ((st = check_pitch("ldx", ldx, width)) != MS_OK) return st;
    if (z && (st = check_pitch("ldz", ldz, width)) != MS_OK) return st;
    if (gate_first && !z) return fail(MS_ERR_NULL, "z is required with gate_first");
    if (rows && (!x || !dy || !dx || (z && !dz)))
        return fail(MS_ERR_NULL, "x, dy and dx are required, and dz with z");
    if ((st = check_aligned({dx, dz, dweight, dbias, workspace})) != MS_OK) return st;
    if ((st = check_element_aligned(io_size(io), {x, z, dy})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {weight, bias})) != MS_OK) return st;
    if (!dweight && !dbias && rows == 0) return MS_OK;
    if ((dweight || dbias) &&
        (st = check_workspace(norm_bwd_ws(a), workspace, workspace_bytes)) != MS_OK)
        return st;
    a.x = x; a.ldx = ldx; a.weight = weight; a.bias = bias; a.z = z; a.ldz = ldz;
    a.center = center; a.gate_first = gate_first; a.dy = dy; a.dx = dx; a.dz = dz;
    a.dweight = dweight; a.dbias = dbias;
    prof_call();
    return launched(launch_norm_bwd(a, io == MS_BF16, workspace, static_cast<hipStream_t>(stream)));
}

size_t ms_verify_drafts_workspace_bytes(int32_t batch, int32_t drafts, int64_t vocab,
                                        int32_t drafted, int32_t io) {
    VerifyArgs a{};
    if (check_verify(a, batch, drafts, vocab, drafted, io) != MS_OK) return (size_t)-1;
    return batch ? verify_ws(a).total : 0;
}

ms_status ms_verify_drafts(const void* logits, int64_t ld, const void* draft_logits, int64_t ldd,
                           const void* drafts_in, int32_t id_bits, const float* uniforms,
                           float scale, int32_t* tokens, int32_t* count, float* logprob,
                           int32_t batch, int32_t drafts, int64_t vocab, int32_t io,
                           void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    VerifyArgs a{};
    ms_status st = check_verify(a, batch, drafts, vocab, draft_logits != nullptr, io);
    if (st != MS_OK) return st;
    if ((st = check_id_bits(id_bits)) != MS_OK) return st;
    if ((st = check_scale(scale, true)) != MS_OK) return st;
    if ((st = check_pitch("ld", ld, vocab)) != MS_OK) return st;
    if (draft_logits && (st = check_pitch("ldd", ldd, vocab)) != MS_OK) return st;
    if (batch == 0) return MS_OK;
    if (!logits || (drafts && !drafts_in) || !uniforms || !tokens || !count || !logprob)
        return fail(MS_ERR_NULL, "logits, drafts, uniforms, tokens, count and logprob are required");
    if ((st = check_element_aligned(io_size(io), {logits, draft_logits})) != MS_OK) return st;
    if ((st = check_element_aligned(id_bits / 8, {drafts_in})) != MS_OK) return st;
    if ((st = check_element_aligned(4, {uniforms, tokens, count, logprob})) != MS_OK) return st;
    if ((st = check_aligned({workspace})) != MS_OK) return st;
    if ((st = check_workspace(verify_ws(a).total, workspace, workspace_bytes)) != MS_OK) return st;
    a.logits = logits; a.ld = ld; a.draft_logits = draft_logits; a.ldd = ldd;
    a.tokens_in = drafts_in; a.wide = id_bits == 64; a.uniforms = uniforms; a.scale = scale;
    a.tokens = tokens; a.count = count; a.logprob = logprob;
    prof_call();
    return launched(launch_verify(a, io == MS_BF16, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
