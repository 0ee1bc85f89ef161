// C-ABI layer of the gated linear recurrence: argument validation and errors.
// Declarations and the contract of every entry point are in include/glr.h.
#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "glr.h"
#include "glr_launch.h"
#include "glr_plan.h"

#define GLR_API extern "C" __attribute__((visibility("default")))

namespace {

using api::Buf;
using api::check_bufs;
using api::check_dtype;
using api::hip_status;
using api::ok;
using api::set_error;

// The products keep every byte count below 2^63 and launches below 2^32
// threads (512 a tile of 64 tokens and 64 channels, 512 for 64 sequences).
kda_status check_sizes(int64_t n_tokens, int32_t D)
{
    if (D < 1) return set_error(KDA_ERR_INVALID_ARG, "D must be >= 1 (got %d)", D);
    if (D >= 1 << 24) return set_error(KDA_ERR_INVALID_ARG, "D must be below 2^24 (got %d)", D);
    if (n_tokens < 0) return set_error(KDA_ERR_INVALID_ARG, "n_tokens must be >= 0");
    if (n_tokens > ((int64_t)1 << 31) - 256)
        return set_error(KDA_ERR_INVALID_ARG, "n_tokens must be at most 2^31 - 256");
    if (n_tokens * D >= (int64_t)1 << 40)
        return set_error(KDA_ERR_INVALID_ARG, "n_tokens * D must be below 2^40");
    if ((n_tokens + 63) / 64 * (((int64_t)D + 63) / 64) >= (int64_t)1 << 22)
        return set_error(KDA_ERR_INVALID_ARG,
                         "the tiles of 64 tokens and 64 channels must be fewer than 2^22");
    return KDA_OK;
}

kda_status check_seqs(int32_t n_seqs, int64_t n_tokens, int32_t D, const int32_t *cu)
{
    if (n_seqs < 0) return set_error(KDA_ERR_INVALID_ARG, "n_seqs must be >= 0 (got %d)", n_seqs);
    if (n_seqs >= 1 << 27) return set_error(KDA_ERR_INVALID_ARG, "n_seqs must be below 2^27 (got %d)", n_seqs);
    if ((int64_t)n_seqs * D >= (int64_t)1 << 40)
        return set_error(KDA_ERR_INVALID_ARG, "n_seqs * D must be below 2^40");
    if (n_seqs == 0 && n_tokens != 0)
        return set_error(KDA_ERR_INVALID_ARG, "n_tokens > 0 with n_seqs == 0");
    if (n_seqs > 0 && !cu && n_tokens % n_seqs)
        return set_error(KDA_ERR_INVALID_ARG,
                         "without cu_seqlens n_tokens (%lld) must be a multiple of n_seqs (%d)",
                         (long long)n_tokens, n_seqs);
    return KDA_OK;
}

size_t kept_bytes(int64_t n_tokens, int32_t D) { return (size_t)glr::tiles_of(n_tokens, glr::kKept) * D * 4; }
size_t fwd_bytes(int64_t n_tokens, int32_t D) { return glr::chain_bytes(glr::tiles_of(n_tokens, glr::kScanTile), D); }

kda_status check_workspace(const void *ws, size_t bytes, size_t need, const char *fn)
{
    if (!need) return KDA_OK;
    if (!ws) return set_error(KDA_ERR_INVALID_ARG, "workspace is NULL");
    if (bytes < need)
        return set_error(KDA_ERR_INVALID_ARG, "workspace_bytes %zu is below the %zu bytes %s gives", bytes,
                         need, fn);
    return KDA_OK;
}

kda_status fwd(const char *fn, glr::Args a, int64_t n_tokens, kda_dtype in_dtype, size_t ws_bytes)
{
    kda_status s;
    if ((s = check_dtype(in_dtype)) != KDA_OK) return s;
    if ((s = check_sizes(n_tokens, a.D)) != KDA_OK) return s;
    if ((s = check_seqs(a.n_seqs, n_tokens, a.D, a.cu_seqlens)) != KDA_OK) return s;
    if (a.n_seqs == 0) return ok();
    const bool tok = n_tokens > 0;
    const size_t ib = in_dtype == KDA_BF16 ? 2 : 4, row = (size_t)n_tokens * a.D;
    const size_t st = (size_t)a.n_seqs * a.D * 4, need = fwd_bytes(n_tokens, a.D);
    if ((s = check_workspace(a.ws, ws_bytes, need, "glr_fwd_workspace_bytes")) != KDA_OK) return s;
    const bool gt = a.gated;
    const Buf bufs[] = {
        {a.x, "x", tok, ib, row * ib, false}, {a.r, "r", tok && gt, ib, row * ib, false},
        {a.i, "i", tok && gt, ib, row * ib, false}, {a.rate, "rate", tok && gt, 4, (size_t)a.D * 4, false},
        {a.g, "g", tok && !gt, 4, row * 4, false}, {a.h0, "h0", false, 4, st, false},
        {a.cu_seqlens, "cu_seqlens", false, 4, ((size_t)a.n_seqs + 1) * 4, false},
        {a.h, "h", false, ib, row * ib, true}, {a.h_T, "h_T", false, 4, st, true},
        {a.kept, "kept", false, 4, kept_bytes(n_tokens, a.D), true},
        {need ? a.ws : nullptr, "workspace", false, 256, need, true}};
    if ((s = check_bufs(bufs, (int)(sizeof(bufs) / sizeof(bufs[0])))) != KDA_OK) return s;
    a.n_tokens = (int32_t)n_tokens;
    a.seqlen = a.cu_seqlens ? 0 : (int32_t)(n_tokens / a.n_seqs);
    a.bf16 = in_dtype == KDA_BF16;
    return hip_status(glr::launch_fwd(a), fn);
}

kda_status bwd(const char *fn, glr::Args a, int64_t n_tokens, kda_dtype in_dtype, size_t ws_bytes)
{
    kda_status s;
    if ((s = check_dtype(in_dtype)) != KDA_OK) return s;
    if ((s = check_sizes(n_tokens, a.D)) != KDA_OK) return s;
    if ((s = check_seqs(a.n_seqs, n_tokens, a.D, a.cu_seqlens)) != KDA_OK) return s;
    const bool tok = n_tokens > 0, gt = a.gated;
    const size_t ib = in_dtype == KDA_BF16 ? 2 : 4, row = (size_t)n_tokens * a.D;
    const size_t st = (size_t)a.n_seqs * a.D * 4, need = glr::GradParts::bytes(n_tokens, a.D);
    if ((s = check_workspace(a.ws, ws_bytes, need, "glr_bwd_workspace_bytes")) != KDA_OK) return s;
    const Buf bufs[] = {
        {a.x, "x", tok, ib, row * ib, false}, {a.r, "r", tok && gt, ib, row * ib, false},
        {a.i, "i", tok && gt, ib, row * ib, false}, {a.rate, "rate", tok && gt, 4, (size_t)a.D * 4, false},
        {a.g, "g", tok && !gt, 4, row * 4, false}, {a.h0, "h0", false, 4, st, false},
        {a.cu_seqlens, "cu_seqlens", false, 4, ((size_t)a.n_seqs + 1) * 4, false},
        {a.kept, "kept", false, 4, kept_bytes(n_tokens, a.D), false}, {a.dh, "dh", tok, ib, row * ib, false},
        {a.dh_T, "dh_T", false, 4, st, false}, {a.dx, "dx", tok, ib, row * ib, true},
        {a.dr, "dr", tok && gt, ib, row * ib, true}, {a.di, "di", tok && gt, ib, row * ib, true},
        {a.drate, "drate", gt, 4, (size_t)a.D * 4, true}, {a.dg, "dg", tok && !gt, 4, row * 4, true},
        {a.dh0, "dh0", false, 4, st, true}, {need ? a.ws : nullptr, "workspace", false, 256, need, true}};
    if ((s = check_bufs(bufs, (int)(sizeof(bufs) / sizeof(bufs[0])))) != KDA_OK) return s;
    a.n_tokens = (int32_t)n_tokens;
    a.seqlen = a.cu_seqlens || !a.n_seqs ? 0 : (int32_t)(n_tokens / a.n_seqs);
    a.bf16 = in_dtype == KDA_BF16;
    return hip_status(glr::launch_bwd(a), fn);
}

glr::Args base(const void *x, const float *h0, const int32_t *cu, int32_t n_seqs, int32_t D, void *ws,
               kda_stream_t stream)
{
    glr::Args a{};
    a.x = x; a.h0 = h0; a.cu_seqlens = cu; a.n_seqs = n_seqs; a.D = D; a.ws = ws;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

kda_status decode(const char *fn, glr::DecodeArgs a, kda_dtype in_dtype)
{
    kda_status s;
    if ((s = check_dtype(in_dtype)) != KDA_OK) return s;
    if (a.N < 0) return set_error(KDA_ERR_INVALID_ARG, "N must be >= 0 (got %d)", a.N);
    if ((s = check_sizes(a.N, a.D)) != KDA_OK) return s;
    if (a.n_slots < 0) return set_error(KDA_ERR_INVALID_ARG, "n_slots must be >= 0 (got %d)", a.n_slots);
    if ((int64_t)a.n_slots * a.D >= (int64_t)1 << 40)
        return set_error(KDA_ERR_INVALID_ARG, "n_slots * D must be below 2^40");
    if (!a.slots && a.N > a.n_slots)
        return set_error(KDA_ERR_INVALID_ARG, "without slots N (%d) must be at most n_slots (%d)", a.N,
                         a.n_slots);
    if (a.N == 0) return ok();
    const bool gt = a.gated;
    const size_t ib = in_dtype == KDA_BF16 ? 2 : 4, row = (size_t)a.N * a.D;
    const Buf bufs[] = {
        {a.x, "x", true, ib, row * ib, false}, {a.r, "r", gt, ib, row * ib, false},
        {a.i, "i", gt, ib, row * ib, false}, {a.rate, "rate", gt, 4, (size_t)a.D * 4, false},
        {a.g, "g", !gt, 4, row * 4, false}, {a.slots, "slots", false, 4, (size_t)a.N * 4, false},
        {a.h, "h", true, ib, row * ib, true},
        {a.S, "S", a.n_slots > 0, 4, (size_t)a.n_slots * a.D * 4, true}};
    if ((s = check_bufs(bufs, (int)(sizeof(bufs) / sizeof(bufs[0])))) != KDA_OK) return s;
    a.bf16 = in_dtype == KDA_BF16;
    return hip_status(glr::launch_decode(a), fn);
}

}  // namespace

GLR_API size_t glr_kept_bytes(int64_t n_tokens, int32_t D)
{
    return check_sizes(n_tokens, D) == KDA_OK ? kept_bytes(n_tokens, D) : 0;
}

GLR_API size_t glr_fwd_workspace_bytes(int64_t n_tokens, int32_t D)
{
    return check_sizes(n_tokens, D) == KDA_OK ? fwd_bytes(n_tokens, D) : 0;
}

GLR_API size_t glr_bwd_workspace_bytes(int64_t n_tokens, int32_t D)
{
    return check_sizes(n_tokens, D) == KDA_OK ? glr::GradParts::bytes(n_tokens, D) : 0;
}

GLR_API kda_status glr_fwd_scan(const void *x, const float *g, const float *h0,
                                const int32_t *cu_seqlens, int32_t n_seqs, int64_t n_tokens,
                                int32_t D, kda_dtype in_dtype, void *h, float *h_T, float *kept,
                                void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    glr::Args a = base(x, h0, cu_seqlens, n_seqs, D, workspace, stream);
    a.g = g; a.h = h; a.h_T = h_T; a.kept = kept;
    return fwd("glr_fwd_scan launch", a, n_tokens, in_dtype, workspace_bytes);
}

GLR_API kda_status glr_fwd_scan_gated(const void *x, const void *r, const void *i, const float *rate,
                                      const float *h0, const int32_t *cu_seqlens, int32_t n_seqs,
                                      int64_t n_tokens, int32_t D, kda_dtype in_dtype, void *h,
                                      float *h_T, float *kept, void *workspace,
                                      size_t workspace_bytes, kda_stream_t stream)
{
    glr::Args a = base(x, h0, cu_seqlens, n_seqs, D, workspace, stream);
    a.gated = true; a.r = r; a.i = i; a.rate = rate; a.h = h; a.h_T = h_T; a.kept = kept;
    return fwd("glr_fwd_scan_gated launch", a, n_tokens, in_dtype, workspace_bytes);
}

GLR_API kda_status glr_bwd_scan(const void *x, const float *g, const float *h0,
                                const int32_t *cu_seqlens, int32_t n_seqs, int64_t n_tokens,
                                int32_t D, kda_dtype in_dtype, const float *kept, const void *dh,
                                const float *dh_T, void *dx, float *dg, float *dh0, void *workspace,
                                size_t workspace_bytes, kda_stream_t stream)
{
    glr::Args a = base(x, h0, cu_seqlens, n_seqs, D, workspace, stream);
    a.g = g; a.kept = const_cast<float *>(kept); a.dh = dh; a.dh_T = dh_T; a.dx = dx; a.dg = dg;
    a.dh0 = dh0;
    return bwd("glr_bwd_scan launch", a, n_tokens, in_dtype, workspace_bytes);
}

GLR_API kda_status glr_bwd_scan_gated(const void *x, const void *r, const void *i, const float *rate,
                                      const float *h0, const int32_t *cu_seqlens, int32_t n_seqs,
                                      int64_t n_tokens, int32_t D, kda_dtype in_dtype,
                                      const float *kept, const void *dh, const float *dh_T, void *dx,
                                      void *dr, void *di, float *drate, float *dh0, void *workspace,
                                      size_t workspace_bytes, kda_stream_t stream)
{
    glr::Args a = base(x, h0, cu_seqlens, n_seqs, D, workspace, stream);
    a.gated = true; a.r = r; a.i = i; a.rate = rate; a.kept = const_cast<float *>(kept); a.dh = dh;
    a.dh_T = dh_T; a.dx = dx; a.dr = dr; a.di = di; a.drate = drate; a.dh0 = dh0;
    return bwd("glr_bwd_scan_gated launch", a, n_tokens, in_dtype, workspace_bytes);
}

GLR_API kda_status glr_decode_step(const void *x, const float *g, float *S, const int32_t *slots,
                                   int32_t n_slots, int32_t N, int32_t D, kda_dtype in_dtype, void *h,
                                   kda_stream_t stream)
{
    glr::DecodeArgs a{};
    a.x = x; a.g = g; a.S = S; a.slots = slots; a.n_slots = n_slots; a.N = N; a.D = D; a.h = h;
    a.stream = static_cast<hipStream_t>(stream);
    return decode("glr_decode_step launch", a, in_dtype);
}

GLR_API kda_status glr_decode_step_gated(const void *x, const void *r, const void *i,
                                         const float *rate, float *S, const int32_t *slots,
                                         int32_t n_slots, int32_t N, int32_t D, kda_dtype in_dtype,
                                         void *h, kda_stream_t stream)
{
    glr::DecodeArgs a{};
    a.gated = true; a.x = x; a.r = r; a.i = i; a.rate = rate; a.S = S; a.slots = slots;
    a.n_slots = n_slots; a.N = N; a.D = D; a.h = h; a.stream = static_cast<hipStream_t>(stream);
    return decode("glr_decode_step_gated launch", a, in_dtype);
}
