/*
 * Gated linear recurrence -- one decaying number per channel, next to the
 * matrix states of Kimi Delta Attention (kda.h) and of the gated delta rule
 * (gdr.h), in the same library.
 *
 * C ABI.  Plain pointers and sizes; no C++ or framework types cross it.
 *
 * What is computed.  Per channel c of a sequence, for every token t
 *
 *     h_t = a_t h_{t-1} + u_t
 *
 * where a_t and u_t come in one of two forms:
 *
 *     plain    a = exp(g),              u = x
 *     gated    a = exp(-rate_c s(r)),   u = sqrt(1 - a^2) s(i) x
 *
 * with s(z) = 1 / (1 + exp(-z)), r and i the pre-activations of a decay gate
 * and an input gate, and rate_c >= 0 one number a channel.  The factor
 * sqrt(1 - a^2) keeps h at u's size whatever the decay; it is formed from
 * exp(g) - 1, so that it keeps its digits at decays near 1.
 *
 * Layouts (all dense, row-major, token-major, no padding; D channels, which
 * need not be a power of two or a multiple of anything):
 *     x, h, r, i     [n_tokens, D]   in_dtype
 *     g              [n_tokens, D]   float32, natural-log decay, g <= 0
 *     rate           [D]             float32, >= 0 and finite
 *     h0, h_T        [n_seqs, D]     float32
 *     kept           [ceil(n_tokens / 32), D] float32
 *     cu_seqlens     int32 [n_seqs + 1] in device memory, cu_seqlens[0] = 0,
 *                    non-decreasing, cu_seqlens[n_seqs] <= n_tokens; NULL:
 *                    n_seqs sequences of n_tokens / n_seqs tokens each
 * h is rounded to in_dtype where it is stored; the recurrence runs in fp32.
 * Rows of tokens behind the last sequence are not read, and in the outputs
 * not written.  A sequence's first token is scaled by sqrt(1 - a^2) like any
 * other.
 *
 * g = -inf is allowed and forgets the state.  g > 0 is computed as given
 * where no product of successive factors overflows.  NaN or an infinity in
 * an input of a token (but g = -inf) may reach any output of its own channel
 * and sequence, and the gradient of rate_c, and none of another's.  Where a
 * gate is so far closed that 1 - a^2 is below fp32's smallest normal number
 * (1.2e-38), u is 0 and the part of the gradients that passes through
 * sqrt(1 - a^2), whose slope is infinite at 0, is taken as 0.
 *
 * Sizes: 1 <= D < 2^24; 0 <= n_seqs < 2^27; 0 <= n_tokens <= 2^31 - 256, and 0 where
 * n_seqs is; n_tokens, n_seqs
 * and (decode) N times D below 2^40, and the number of (64 tokens, 64
 * channels) tiles below 2^22.  in_dtype KDA_BF16 or KDA_F32.
 *
 * Alignment: every tensor to its own elements, workspaces to 256 bytes.
 * (Pairs of channels are read at once where D and the addresses allow.)
 *
 * Ownership, errors and concurrency are those of kda.h: the caller owns
 * every buffer, nothing is allocated or synchronised, argument problems are
 * reported as a kda_status (kda_last_error has the message) before anything
 * is launched, and cu_seqlens and slots that break their contract change
 * results, never the addresses touched.  Two calls in flight need separate
 * workspaces: in one that something else writes meanwhile a call finds any
 * states, or NaN where a wait for one gives up after a second or more.
 *
 * Results do not depend on the order in which workgroups run, and a call
 * repeated gives the same bits.  Their last bits (within the same error bounds)
 * do depend on the form that is taken by sizes and alignment and, gated, on
 * whether all rates of the 64 or 128 channels that a wave takes at once are at
 * most 0.69.
 */
#ifndef GLR_H
#define GLR_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * glr_fwd_scan, glr_fwd_scan_gated -- the recurrence over a packed batch.
 *
 * Writes h for every token (skipped when NULL) and the state after each
 * sequence's last token to h_T (skipped when NULL), starting from h0 (zeros
 * when NULL).  An empty sequence gives h_T = h0.  kept, when not NULL, gets
 * what the backward wants: the state before every 32nd token of the batch
 * (glr_kept_bytes bytes).  The workspace holds glr_fwd_workspace_bytes bytes
 * and may be NULL where that is 0.
 */
size_t glr_kept_bytes(int64_t n_tokens, int32_t D);
size_t glr_fwd_workspace_bytes(int64_t n_tokens, int32_t D);
kda_status glr_fwd_scan(const void *x, const float *g, const float *h0, const int32_t *cu_seqlens,
                        int32_t n_seqs, int64_t n_tokens, int32_t D, kda_dtype in_dtype, void *h,
                        float *h_T, float *kept, void *workspace, size_t workspace_bytes,
                        kda_stream_t stream);
kda_status glr_fwd_scan_gated(const void *x, const void *r, const void *i, const float *rate,
                              const float *h0, const int32_t *cu_seqlens, int32_t n_seqs,
                              int64_t n_tokens, int32_t D, kda_dtype in_dtype, void *h, float *h_T,
                              float *kept, void *workspace, size_t workspace_bytes,
                              kda_stream_t stream);

/*
 * glr_bwd_scan, glr_bwd_scan_gated -- gradients of the above.
 *
 * dh is h's cotangent (in_dtype), dh_T the final states' (float32, or NULL
 * for zero).  kept is what the forward of the same inputs left, or NULL: it
 * is formed again then.  Writes dx (gated: dr, di too) in in_dtype, dg in
 * float32, drate [D] in float32 and dh0 [n_seqs, D] in float32 (skipped when
 * NULL).  The workspace (required where it is not 0 bytes) holds
 * glr_bwd_workspace_bytes bytes.  An empty sequence gives dh0 = dh_T.
 */
size_t glr_bwd_workspace_bytes(int64_t n_tokens, int32_t D);
kda_status glr_bwd_scan(const void *x, const float *g, const float *h0, const int32_t *cu_seqlens,
                        int32_t n_seqs, int64_t n_tokens, int32_t D, kda_dtype in_dtype,
                        const float *kept, const void *dh, const float *dh_T, void *dx, float *dg,
                        float *dh0, void *workspace, size_t workspace_bytes, kda_stream_t stream);
kda_status glr_bwd_scan_gated(const void *x, const void *r, const void *i, const float *rate,
                              const float *h0, const int32_t *cu_seqlens, int32_t n_seqs,
                              int64_t n_tokens, int32_t D, kda_dtype in_dtype, const float *kept,
                              const void *dh, const float *dh_T, void *dx, void *dr, void *di,
                              float *drate, float *dh0, void *workspace, size_t workspace_bytes,
                              kda_stream_t stream);

/*
 * glr_decode_step, glr_decode_step_gated -- one token for each of N requests,
 * states in a pool.
 *
 * x, r, i, g, h [N, D].  S is a pool of n_slots states [n_slots, D], updated
 * IN PLACE: request n reads and writes the state slots[n] (slots NULL: state
 * n, N <= n_slots).  A slot outside [0, n_slots) marks a padded row of the
 * batch: its h row is written with zeros and no state is touched.  The slots
 * of a call must differ from one another: two requests of one slot race,
 * which leaves that state and both h rows undefined and touches no other
 * memory.
 */
kda_status glr_decode_step(const void *x, const float *g, float *S, const int32_t *slots,
                           int32_t n_slots, int32_t N, int32_t D, kda_dtype in_dtype, void *h,
                           kda_stream_t stream);
kda_status glr_decode_step_gated(const void *x, const void *r, const void *i, const float *rate,
                                 float *S, const int32_t *slots, int32_t n_slots, int32_t N,
                                 int32_t D, kda_dtype in_dtype, void *h, kda_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GLR_H */
