// C-ABI layer of the gated delta rule: argument validation and errors.
// Declarations and the contract of every entry point are in include/gdr.h.
#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "gdr.h"
#include "gdr_launch.h"

#define GDR_API extern "C" __attribute__((visibility("default")))

namespace gdr {

// Matrix-core chunks for bf16 (or 8-bit) inputs and heads of 64 or 128;
// everything else token by token in fp32.
static bool chunked(int dk, int dv, bool bf16) { return bf16 && dk >= 64 && dv >= 64; }

int bwd_chunk(int dk, int dv, bool bf16) { return chunked(dk, dv, bf16) ? 64 : kRecurrentChunk; }

static hipError_t launch_fwd(const Args &a)
{
    return chunked(a.dk, a.dv, a.in == In::BF16) ? launch_chunk_fwd(a) : launch_recurrent_fwd(a);
}

static hipError_t launch_bwd(const Args &a)
{
    const bool bf16 = a.in != In::F32;
    hipError_t e;
    if (chunked(a.dk, a.dv, bf16)) {
        if ((e = launch_chunk_keep_sweep(a)) != hipSuccess || a.seq.n_tokens == 0) return e;
        return launch_chunk_grad(a);
    }
    if ((e = launch_recurrent_keep_sweep(a)) != hipSuccess || a.seq.n_tokens == 0) return e;
    return launch_grad32(a);
}

}  // namespace gdr

namespace {

using api::Buf;
using api::check_bufs;
using api::check_dtype;
using api::hip_status;
using api::ok;
using api::round256;
using api::set_error;

bool head_dim_ok(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

kda_status check_heads(int32_t Hk, int32_t Hv, int32_t dk, int32_t dv)
{
    if (Hk < 1) return set_error(KDA_ERR_INVALID_ARG, "H_k must be >= 1 (got %d)", Hk);
    if (Hv < 1 || Hv % Hk)
        return set_error(KDA_ERR_INVALID_ARG, "H_v (%d) must be a positive multiple of H_k (%d)",
                         Hv, Hk);
    if (!head_dim_ok(dk) || !head_dim_ok(dv))
        return set_error(KDA_ERR_UNSUPPORTED, "d_k and d_v must be 16, 32, 64 or 128 (got %d, %d)",
                         dk, dv);
    if ((int64_t)Hv * (dk > dv ? dk : dv) >= ((int64_t)1 << 22))
        return set_error(KDA_ERR_INVALID_ARG, "H_v * d must be below 2^22 (64 rows of a tensor must stay "
                                              "below 2^31 bytes)");
    return KDA_OK;
}

kda_status check_tokens(int64_t n_tokens)
{
    if (n_tokens < 0) return set_error(KDA_ERR_INVALID_ARG, "n_tokens must be >= 0");
    if (n_tokens > ((int64_t)1 << 31) - 64)
        return set_error(KDA_ERR_INVALID_ARG, "n_tokens must be at most 2^31 - 64");
    return KDA_OK;
}

kda_status check_seqs(int32_t n_seqs, int64_t n_tokens, const int32_t *cu)
{
    kda_status s;
    if (n_seqs < 0) return set_error(KDA_ERR_INVALID_ARG, "n_seqs must be >= 0 (got %d)", n_seqs);
    if ((s = check_tokens(n_tokens)) != KDA_OK) return s;
    if (n_seqs == 0 && n_tokens != 0)
        return set_error(KDA_ERR_INVALID_ARG, "n_tokens > 0 with n_seqs == 0");
    if (reinterpret_cast<uintptr_t>(cu) % 4)
        return set_error(KDA_ERR_INVALID_ARG, "cu_seqlens is not 4-byte aligned");
    if (n_seqs > 0 && !cu && n_tokens % n_seqs)
        return set_error(KDA_ERR_INVALID_ARG,
                         "without cu_seqlens n_tokens (%lld) must be a multiple of n_seqs (%d)",
                         (long long)n_tokens, n_seqs);
    return KDA_OK;
}

// Launches must stay below 2^32 threads.  The widest ones: 2048 threads a
// (sequence, value head) chain, 1024 a decoded head, 512 a 64-token chunk and
// key head (256 a 32-token one).  Checked before anything is launched.
kda_status check_chains(int64_t chains, const char *what)
{
    if (chains >= (int64_t)1 << 21)
        return set_error(KDA_ERR_INVALID_ARG, "%s * H_v must be below 2^21", what);
    return KDA_OK;
}

gdr::Args base_args(const float *g, const float *beta, const float *S0, const int32_t *cu,
                    int32_t n_seqs, int64_t n_tokens, int32_t Hk, int32_t Hv, int32_t dk,
                    int32_t dv, float scale, void *stream)
{
    gdr::Args a{};
    a.g = g; a.beta = beta; a.S0 = S0;
    a.seq.cu_seqlens = cu; a.seq.n_seqs = n_seqs; a.seq.n_tokens = (int32_t)n_tokens;
    a.seq.seqlen = cu ? 0 : (int32_t)(n_tokens / n_seqs);
    a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv; a.scale = scale;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

struct Parts {
    size_t state, rows;                  // bytes of each of the two state and two row arrays
    size_t total() const { return 2 * state + 2 * rows; }
};
Parts bwd_parts(int32_t n_seqs, int64_t n_tokens, int32_t Hv, int32_t dk, int32_t dv, bool bf16)
{
    const size_t slots = (size_t)gdr::bwd_slots(n_seqs, n_tokens, gdr::bwd_chunk(dk, dv, bf16));
    return Parts{round256(slots * Hv * dk * dv * 4), round256((size_t)n_tokens * Hv * dv * 4)};
}

// exponent bytes of rows of d channels
size_t exp_bytes(size_t rows, int32_t d) { return rows * (d / (d < 32 ? d : 32)); }

kda_status bwd_impl(const char *fn, const void *q, const uint8_t *qe, const void *k,
                    const uint8_t *ke, const void *v, const uint8_t *ve, const float *g,
                    const float *beta, const float *S0, const int32_t *cu, int32_t n_seqs,
                    int64_t n_tokens, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, float scale,
                    gdr::In in, const void *dO, const float *dS_T, void *dq, void *dkey,
                    void *dval, float *dg, float *dbeta, float *dS0, void *ws, size_t ws_bytes,
                    kda_stream_t stream)
{
    kda_status s;
    if ((s = check_heads(Hk, Hv, dk, dv)) != KDA_OK) return s;
    if ((s = check_seqs(n_seqs, n_tokens, cu)) != KDA_OK) return s;
    if ((s = check_chains((int64_t)n_seqs * Hv, "n_seqs")) != KDA_OK) return s;
    // the chunk form deals a key head's workgroups out in rounds of eight (2048
    // threads a chain at d_v = 128, half of that at 64)
    if (gdr::chunked(dk, dv, in != gdr::In::F32) && dv == 128 &&
        ((int64_t)n_seqs * Hk + 7) / 8 * 8 * (Hv / Hk) >= (int64_t)1 << 21)
        return set_error(KDA_ERR_INVALID_ARG,
                         "n_seqs * H_k rounded up to a multiple of 8, times H_v / H_k, must be below 2^21");
    if (gdr::bwd_slots(n_seqs, n_tokens, gdr::bwd_chunk(dk, dv, in != gdr::In::F32)) * Hk >= (int64_t)1 << 23)
        return set_error(KDA_ERR_INVALID_ARG, "too many chunks times H_k for one launch (2^23)");
    if (n_seqs == 0) return ok();
    const bool e8 = in == gdr::In::E4M3, tok = n_tokens > 0;
    const size_t ib = in == gdr::In::F32 ? 4 : 2, qb = e8 ? 1 : ib;
    const size_t rk = (size_t)n_tokens * Hk, rv = (size_t)n_tokens * Hv;
    const size_t st = (size_t)n_seqs * Hv * dk * dv * 4;
    const Parts pt = bwd_parts(n_seqs, n_tokens, Hv, dk, dv, in != gdr::In::F32);
    if (!ws) return set_error(KDA_ERR_INVALID_ARG, "workspace is NULL");
    if (ws_bytes < pt.total())
        return set_error(KDA_ERR_INVALID_ARG,
                         "workspace_bytes %zu is below the %zu bytes gdr_bwd_workspace_bytes gives",
                         ws_bytes, pt.total());
    const Buf bufs[] = {
        {q, e8 ? "q8" : "q", tok, 16, rk * dk * qb, false}, {k, e8 ? "k8" : "k", tok, 16, rk * dk * qb, false},
        {v, e8 ? "v8" : "v", tok, 16, rv * dv * qb, false},
        {qe, "qe", tok && e8, 1, e8 ? exp_bytes(rk, dk) : 0, false},
        {ke, "ke", tok && e8, 1, e8 ? exp_bytes(rk, dk) : 0, false},
        {ve, "ve", tok && e8, 1, e8 ? exp_bytes(rv, dv) : 0, false},
        {g, "g", tok, 4, rv * 4, false}, {beta, "beta", tok, 4, rv * 4, false},
        {S0, "S0", false, 16, st, false}, {dO, "dO", tok, 16, rv * dv * ib, false},
        {dS_T, "dS_T", false, 16, st, false}, {cu, "cu_seqlens", false, 4, ((size_t)n_seqs + 1) * 4, false},
        {dq, "dq", tok, 16, rk * dk * ib, true}, {dkey, "dk", tok, 16, rk * dk * ib, true},
        {dval, "dv", tok, 16, rv * dv * ib, true}, {dg, "dg", tok, 4, rv * 4, true},
        {dbeta, "dbeta", tok, 4, rv * 4, true}, {dS0, "dS0", false, 16, st, true},
        {ws, "workspace", true, 256, pt.total(), true}};
    if ((s = check_bufs(bufs, (int)(sizeof(bufs) / sizeof(bufs[0])))) != KDA_OK) return s;
    gdr::Args a = base_args(g, beta, S0, cu, n_seqs, n_tokens, Hk, Hv, dk, dv, scale, stream);
    a.q = q; a.k = k; a.v = v; a.qe = qe; a.ke = ke; a.ve = ve; a.in = in;
    a.dO = dO; a.dS_T = dS_T;
    a.dq = dq; a.dkey = dkey; a.dval = dval; a.dg = dg; a.dbeta = dbeta; a.dS0 = dS0;
    char *w = static_cast<char *>(ws);
    a.Sc = reinterpret_cast<float *>(w);
    a.Lc = reinterpret_cast<float *>(w + pt.state);
    a.R = reinterpret_cast<float *>(w + 2 * pt.state);
    a.Ub = reinterpret_cast<float *>(w + 2 * pt.state + pt.rows);
    return hip_status(gdr::launch_bwd(a), fn);
}

}  // namespace

GDR_API kda_status gdr_fwd_chunked(const void *q, const void *k, const void *v, const float *g,
                                   const float *beta, const float *S0, const int32_t *cu_seqlens,
                                   int32_t n_seqs, int64_t n_tokens, int32_t H_k, int32_t H_v,
                                   int32_t d_k, int32_t d_v, float scale, kda_dtype in_dtype,
                                   void *o, float *S_T, kda_stream_t stream)
{
    kda_status s;
    if ((s = check_dtype(in_dtype)) != KDA_OK) return s;
    if ((s = check_heads(H_k, H_v, d_k, d_v)) != KDA_OK) return s;
    if ((s = check_seqs(n_seqs, n_tokens, cu_seqlens)) != KDA_OK) return s;
    if ((s = check_chains((int64_t)n_seqs * H_v, "n_seqs")) != KDA_OK) return s;
    if (n_seqs == 0) return ok();
    const bool tok = n_tokens > 0;
    const size_t ib = in_dtype == KDA_BF16 ? 2 : 4;
    const size_t rk = (size_t)n_tokens * H_k, rv = (size_t)n_tokens * H_v;
    const size_t st = (size_t)n_seqs * H_v * d_k * d_v * 4;
    const Buf bufs[] = {
        {q, "q", tok, 16, rk * d_k * ib, false}, {k, "k", tok, 16, rk * d_k * ib, false},
        {v, "v", tok, 16, rv * d_v * ib, false}, {g, "g", tok, 4, rv * 4, false},
        {beta, "beta", tok, 4, rv * 4, false}, {S0, "S0", false, 16, st, false},
        {cu_seqlens, "cu_seqlens", false, 4, ((size_t)n_seqs + 1) * 4, false},
        {o, "o", tok, 16, rv * d_v * ib, true}, {S_T, "S_T", false, 16, st, true}};
    if ((s = check_bufs(bufs, (int)(sizeof(bufs) / sizeof(bufs[0])))) != KDA_OK) return s;
    gdr::Args a = base_args(g, beta, S0, cu_seqlens, n_seqs, n_tokens, H_k, H_v, d_k, d_v, scale,
                            stream);
    a.q = q; a.k = k; a.v = v; a.in = in_dtype == KDA_BF16 ? gdr::In::BF16 : gdr::In::F32;
    a.o = o; a.S_T = S_T;
    return hip_status(gdr::launch_fwd(a), "gdr_fwd_chunked launch");
}

GDR_API kda_status gdr_decode_step(const void *q, const void *k, const void *v, const float *g,
                                   const float *beta, float *S, const int32_t *slots,
                                   int32_t n_slots, int32_t N, int32_t H_k, int32_t H_v,
                                   int32_t d_k, int32_t d_v, float scale, kda_dtype in_dtype,
                                   void *o, kda_stream_t stream)
{
    kda_status s;
    if ((s = check_dtype(in_dtype)) != KDA_OK) return s;
    if ((s = check_heads(H_k, H_v, d_k, d_v)) != KDA_OK) return s;
    if (N < 0) return set_error(KDA_ERR_INVALID_ARG, "N must be >= 0 (got %d)", N);
    if ((s = check_chains((int64_t)N * H_v, "N")) != KDA_OK) return s;
    if (n_slots < 0) return set_error(KDA_ERR_INVALID_ARG, "n_slots must be >= 0 (got %d)", n_slots);
    if (!slots && N > n_slots)
        return set_error(KDA_ERR_INVALID_ARG, "without slots N (%d) must be at most n_slots (%d)", N,
                         n_slots);
    if (N == 0) return ok();
    const size_t ib = in_dtype == KDA_BF16 ? 2 : 4, rk = (size_t)N * H_k, rv = (size_t)N * H_v;
    const Buf bufs[] = {
        {q, "q", true, 16, rk * d_k * ib, false}, {k, "k", true, 16, rk * d_k * ib, false},
        {v, "v", true, 16, rv * d_v * ib, false}, {g, "g", true, 4, rv * 4, false},
        {beta, "beta", true, 4, rv * 4, false}, {slots, "slots", false, 4, (size_t)N * 4, false},
        {o, "o", true, 16, rv * d_v * ib, true},
        {S, "S", n_slots > 0, 16, (size_t)n_slots * H_v * d_k * d_v * 4, true}};
    if ((s = check_bufs(bufs, (int)(sizeof(bufs) / sizeof(bufs[0])))) != KDA_OK) return s;
    gdr::DecodeArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S = S; a.slots = slots;
    a.n_slots = n_slots; a.N = N; a.Hk = H_k; a.Hv = H_v; a.dk = d_k; a.dv = d_v; a.scale = scale;
    a.bf16 = in_dtype == KDA_BF16; a.o = o; a.stream = static_cast<hipStream_t>(stream);
    return hip_status(gdr::launch_decode(a), "gdr_decode_step launch");
}

GDR_API size_t gdr_bwd_workspace_bytes(int32_t n_seqs, int64_t n_tokens, int32_t H_k, int32_t H_v,
                                       int32_t d_k, int32_t d_v, kda_dtype in_dtype)
{
    if (check_dtype(in_dtype) != KDA_OK || check_heads(H_k, H_v, d_k, d_v) != KDA_OK ||
        n_seqs <= 0 || check_tokens(n_tokens) != KDA_OK)
        return 0;
    return bwd_parts(n_seqs, n_tokens, H_v, d_k, d_v, in_dtype == KDA_BF16).total();
}

GDR_API kda_status gdr_bwd_chunked(const void *q, const void *k, const void *v, const float *g,
                                   const float *beta, const float *S0, const int32_t *cu_seqlens,
                                   int32_t n_seqs, int64_t n_tokens, int32_t H_k, int32_t H_v,
                                   int32_t d_k, int32_t d_v, float scale, kda_dtype in_dtype,
                                   const void *dO, const float *dS_T, void *dq, void *dk, void *dv,
                                   float *dg, float *dbeta, float *dS0, void *workspace,
                                   size_t workspace_bytes, kda_stream_t stream)
{
    kda_status s;
    if ((s = check_dtype(in_dtype)) != KDA_OK) return s;
    return bwd_impl("gdr_bwd_chunked launch", q, nullptr, k, nullptr, v, nullptr, g, beta, S0,
                    cu_seqlens, n_seqs, n_tokens, H_k, H_v, d_k, d_v, scale,
                    in_dtype == KDA_BF16 ? gdr::In::BF16 : gdr::In::F32, dO, dS_T, dq, dk, dv, dg,
                    dbeta, dS0, workspace, workspace_bytes, stream);
}

GDR_API kda_status gdr_bwd_chunked_saved8(
    const uint8_t *q8, const uint8_t *qe, const uint8_t *k8, const uint8_t *ke, const uint8_t *v8,
    const uint8_t *ve, const float *g, const float *beta, const float *S0,
    const int32_t *cu_seqlens, int32_t n_seqs, int64_t n_tokens, int32_t H_k, int32_t H_v,
    int32_t d_k, int32_t d_v, float scale, const void *dO, const float *dS_T, void *dq, void *dk,
    void *dv, float *dg, float *dbeta, float *dS0, void *workspace, size_t workspace_bytes,
    kda_stream_t stream)
{
    return bwd_impl("gdr_bwd_chunked_saved8 launch", q8, qe, k8, ke, v8, ve, g, beta, S0,
                    cu_seqlens, n_seqs, n_tokens, H_k, H_v, d_k, d_v, scale, gdr::In::E4M3, dO,
                    dS_T, dq, dk, dv, dg, dbeta, dS0, workspace, workspace_bytes, stream);
}

namespace {

kda_status check8(const void *q, const void *k, const void *v, const uint8_t *q8, const uint8_t *qe,
                  const uint8_t *k8, const uint8_t *ke, const uint8_t *v8, const uint8_t *ve,
                  int64_t n_tokens, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, bool save)
{
    kda_status s;
    if ((s = check_heads(Hk, Hv, dk, dv)) != KDA_OK) return s;
    if ((s = check_tokens(n_tokens)) != KDA_OK) return s;
    if (n_tokens == 0) return ok();
    const size_t rk = (size_t)n_tokens * Hk, rv = (size_t)n_tokens * Hv;
    const Buf bufs[] = {
        {q, "q", true, 16, rk * dk * 2, !save}, {k, "k", true, 16, rk * dk * 2, !save},
        {v, "v", true, 16, rv * dv * 2, !save}, {q8, "q8", true, 16, rk * dk, save},
        {k8, "k8", true, 16, rk * dk, save}, {v8, "v8", true, 16, rv * dv, save},
        {qe, "qe", true, 1, exp_bytes(rk, dk), save}, {ke, "ke", true, 1, exp_bytes(rk, dk), save},
        {ve, "ve", true, 1, exp_bytes(rv, dv), save}};
    return check_bufs(bufs, 9);
}

gdr::Kept8 kept8(const void *q, const void *k, const void *v, const uint8_t *q8, const uint8_t *qe,
                 const uint8_t *k8, const uint8_t *ke, const uint8_t *v8, const uint8_t *ve,
                 int64_t n_tokens, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv)
{
    const auto mut = [](const uint8_t *p) { return const_cast<uint8_t *>(p); };     // read only when loading
    const int64_t rk = n_tokens * Hk * dk / 8, rv = n_tokens * Hv * dv / 8;
    const int lk = dk < 32 ? dk / 8 : 4, lv = dv < 32 ? dv / 8 : 4;
    return gdr::Kept8{{q, k, v}, {mut(q8), mut(k8), mut(v8)}, {mut(qe), mut(ke), mut(ve)},
                      {rk, rk, rv}, {lk, lk, lv}, {}};
}

}  // namespace

GDR_API kda_status gdr_save8(const void *q, const void *k, const void *v, int64_t n_tokens,
                             int32_t H_k, int32_t H_v, int32_t d_k, int32_t d_v, uint8_t *q8,
                             uint8_t *qe, uint8_t *k8, uint8_t *ke, uint8_t *v8, uint8_t *ve,
                             kda_stream_t stream)
{
    kda_status s = check8(q, k, v, q8, qe, k8, ke, v8, ve, n_tokens, H_k, H_v, d_k, d_v, true);
    if (s != KDA_OK || n_tokens == 0) return s;
    return hip_status(gdr::launch_save8(kept8(q, k, v, q8, qe, k8, ke, v8, ve, n_tokens, H_k, H_v, d_k, d_v),
                                        static_cast<hipStream_t>(stream)), "gdr_save8 launch");
}

GDR_API kda_status gdr_load8(const uint8_t *q8, const uint8_t *qe, const uint8_t *k8,
                             const uint8_t *ke, const uint8_t *v8, const uint8_t *ve,
                             int64_t n_tokens, int32_t H_k, int32_t H_v, int32_t d_k, int32_t d_v,
                             void *q, void *k, void *v, kda_stream_t stream)
{
    kda_status s = check8(q, k, v, q8, qe, k8, ke, v8, ve, n_tokens, H_k, H_v, d_k, d_v, false);
    if (s != KDA_OK || n_tokens == 0) return s;
    return hip_status(gdr::launch_load8(kept8(q, k, v, q8, qe, k8, ke, v8, ve, n_tokens, H_k, H_v, d_k, d_v),
                                        static_cast<hipStream_t>(stream)), "gdr_load8 launch");
}
