/*
 * Gated delta rule -- the recurrence with one decay per head and token, next
 * to Kimi Delta Attention's per-channel decay (kda.h), in the same library.
 *
 * C ABI.  Plain pointers and sizes; no C++ or framework types cross it.
 *
 * What is computed.  Per value head, a d_k x d_v state S (rows = key
 * channels); for every token t
 *
 *     S'  = exp(g_t) S_{t-1}
 *     u_t = beta_t (v_t - S'^T k_t)
 *     S_t = S' + k_t u_t^T
 *     o_t = scale S_t^T q_t
 *
 * This is KDA's recurrence with a scalar in place of the channel-wise decay
 * (the Kimi K3 architecture walkthrough, mhpq.cn/news/56770, "KDA 到底在算
 * 什么", names it as Gated DeltaNet), with three things KDA's calls do not
 * have: the decay has no lower bound, an output scale, and key heads shared
 * by groups of value heads: value head h reads q, k of key head
 * h / (H_v / H_k).
 *
 * Layouts (all dense, row-major, token-major, no padding):
 *     q, k    [n_tokens, H_k, d_k]    in_dtype
 *     v, o    [n_tokens, H_v, d_v]    in_dtype
 *     g       [n_tokens, H_v]         float32, natural-log decay, g <= 0
 *     beta    [n_tokens, H_v]         float32
 *     S0, S_T [n_seqs, H_v, d_k, d_v] float32
 *     cu_seqlens  int32 [n_seqs + 1] in device memory, cu_seqlens[0] = 0,
 *                 non-decreasing, cu_seqlens[n_seqs] = n_tokens; NULL: n_seqs
 *                 sequences of n_tokens / n_seqs tokens each
 * g = -inf is allowed and forgets the state (every g below -1e4 counts as
 * -1e4, whose exponential is 0).  g > 0 is computed as given where nothing
 * overflows.  NaN or an infinity in g (but -inf), beta, q, k, v or dO of a
 * token, or in a state or its cotangent, may reach any output of its own
 * sequence and value head (from q and k: of the value heads of their key
 * head), and dq and dk of that key head, and none of another's.  Tokens before
 * it in its chunk of 64 are among them: the chunk's products multiply what the
 * mask leaves out by zero, and zero times such a value is NaN.  Inside a chunk
 * the factors exp(G_i - G_j) of the log-decay's cumulative sums are formed
 * from their differences, so no
 * decay, however fast, overflows.
 *
 * Sizes: d_k, d_v in {16, 32, 64, 128}, independently; 1 <= H_k, H_v a
 * multiple of H_k, H_v * max(d_k, d_v) < 2^22; 0 <= n_tokens <= 2^31 - 64;
 * n_seqs * H_v (decode: N * H_v) < 2^21.  The backward also wants fewer than
 * 2^23 (chunk of 64 tokens, key head) pairs (32 tokens in the fp32 form), and
 * from bf16 or 8-bit inputs with d_k >= 64, d_v = 128 counts n_seqs * H_k
 * rounded up to a multiple of 8 against the 2^21.
 * in_dtype KDA_BF16 or KDA_F32.
 *
 * Alignment (bytes): q, k, v, o, dO, dq, dk, dv: eight elements of bf16 and
 * four of fp32 (16 bytes); g, beta, dg, dbeta, cu_seqlens, slots: 4; states
 * and their gradients: 16.  Any slice of a contiguous tensor along its token
 * (or sequence) axis satisfies these.
 *
 * Ownership, errors and concurrency are those of kda.h: the caller owns
 * every buffer, nothing is allocated or synchronised, argument problems are
 * reported as a kda_status (kda_last_error has the message) before anything
 * is launched, and cu_seqlens and slots that break their contract change
 * results, never the addresses touched: entries of cu_seqlens count as the
 * nearest of 0 .. n_tokens, and a sequence that ends before it starts as
 * empty.  Rows of tokens that no sequence has (behind a last entry below
 * n_tokens) are not read, and in the outputs not written.
 */
#ifndef GDR_H
#define GDR_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdr_fwd_chunked -- the recurrence over a packed batch of sequences.
 *
 * Writes o for every token and the state after each sequence's last token
 * to S_T (skipped when NULL), starting from S0 (zeros when NULL).  An empty
 * sequence gives S_T = S0.  o may be NULL iff n_tokens == 0.
 */
kda_status gdr_fwd_chunked(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, const float *S0, const int32_t *cu_seqlens,
                           int32_t n_seqs, int64_t n_tokens, int32_t H_k, int32_t H_v,
                           int32_t d_k, int32_t d_v, float scale, kda_dtype in_dtype, void *o,
                           float *S_T, kda_stream_t stream);

/*
 * gdr_decode_step -- one token for each of N requests, states in a pool.
 *
 * q, k [N, H_k, d_k]; v, o [N, H_v, d_v]; g, beta [N, H_v].  S is a pool of
 * n_slots states [n_slots, H_v, d_k, d_v], updated IN PLACE: request n reads
 * and writes the state slots[n] (slots NULL: state n, N <= n_slots).  A slot
 * outside [0, n_slots) marks a padded row of the batch: its o row is written
 * with zeros and no state is touched.  The slots of a call must differ from
 * one another: two requests of one slot race, which leaves that state and both
 * o rows undefined (the state may hold elements of either, or of one computed
 * from the other's) and touches no other memory.
 */
kda_status gdr_decode_step(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, float *S, const int32_t *slots, int32_t n_slots,
                           int32_t N, int32_t H_k, int32_t H_v, int32_t d_k, int32_t d_v,
                           float scale, kda_dtype in_dtype, void *o, kda_stream_t stream);

/*
 * gdr_bwd_chunked -- gradients of gdr_fwd_chunked.
 *
 * dO is o's cotangent (in_dtype), dS_T the final states' (float32, or NULL
 * for zero).  Writes dq, dk [n_tokens, H_k, d_k] (summed over the value heads
 * that share a key head) and dv [n_tokens, H_v, d_v] in in_dtype, dg and
 * dbeta [n_tokens, H_v] in float32, and dS0 [n_seqs, H_v, d_k, d_v] in
 * float32 (skipped when NULL).  Results do not depend on the order in which
 * workgroups run.  The workspace (required, 256-byte aligned) holds
 * gdr_bwd_workspace_bytes bytes: states and their cotangents at the chunk
 * borders and two rows per token and head.  Two calls in flight need
 * separate workspaces.
 */
size_t gdr_bwd_workspace_bytes(int32_t n_seqs, int64_t n_tokens, int32_t H_k, int32_t H_v,
                               int32_t d_k, int32_t d_v, kda_dtype in_dtype);
kda_status gdr_bwd_chunked(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, const float *S0, const int32_t *cu_seqlens,
                           int32_t n_seqs, int64_t n_tokens, int32_t H_k, int32_t H_v,
                           int32_t d_k, int32_t d_v, float scale, kda_dtype in_dtype,
                           const void *dO, const float *dS_T, void *dq, void *dk, void *dv,
                           float *dg, float *dbeta, float *dS0, void *workspace,
                           size_t workspace_bytes, kda_stream_t stream);

/*
 * Inputs kept in 8 bits between the passes (bf16 q, k, v).
 *
 * Each head row of d channels is cut into blocks of min(32, d); a block is
 * held as one exponent byte e and its elements as e4m3 bytes x, standing for
 * x 2^(e - 127), with e - 127 the smallest power that brings the block's
 * largest finite magnitude to 448 or less, within [-110, 119] (elements are
 * rounded to nearest even; below the range they lose bits towards zero,
 * above it they stop at 448).  Infinities and NaN become NaN.  The
 * values so kept are bf16 values, so the gradients that
 * gdr_bwd_chunked_saved8 forms from them are those that gdr_bwd_chunked
 * forms from gdr_load8's output, bit for bit.  Against the gradients at the
 * inputs themselves the three roundings move dq, dk and dv by about 4% of
 * their norms and dg and dbeta by 4 to 6% (unit q and k, normal v; each input
 * moves by 2.7% of its own).  What is kept shrinks from 2 to 1 + 1/32 bytes an
 * element: 0.13 GB for 16384 tokens of 16 + 16 + 32 heads of 128, beside the
 * 1.6 GB of workspace that the backward takes while it runs.
 *
 * q8, k8 [n_tokens, H_k, d_k] and v8 [n_tokens, H_v, d_v] bytes (16-byte
 * aligned); qe, ke [n_tokens, H_k, d_k / min(32, d_k)] and ve likewise, bytes.
 */
kda_status gdr_save8(const void *q, const void *k, const void *v, int64_t n_tokens, int32_t H_k,
                     int32_t H_v, int32_t d_k, int32_t d_v, uint8_t *q8, uint8_t *qe,
                     uint8_t *k8, uint8_t *ke, uint8_t *v8, uint8_t *ve, kda_stream_t stream);
kda_status gdr_load8(const uint8_t *q8, const uint8_t *qe, const uint8_t *k8, const uint8_t *ke,
                     const uint8_t *v8, const uint8_t *ve, int64_t n_tokens, int32_t H_k,
                     int32_t H_v, int32_t d_k, int32_t d_v, void *q, void *k, void *v,
                     kda_stream_t stream);
/* gdr_bwd_chunked with in_dtype KDA_BF16 and q, k, v as gdr_save8 left them
 * (workspace: gdr_bwd_workspace_bytes with KDA_BF16). */
kda_status gdr_bwd_chunked_saved8(const uint8_t *q8, const uint8_t *qe, const uint8_t *k8,
                                  const uint8_t *ke, const uint8_t *v8, const uint8_t *ve,
                                  const float *g, const float *beta, const float *S0,
                                  const int32_t *cu_seqlens, int32_t n_seqs, int64_t n_tokens,
                                  int32_t H_k, int32_t H_v, int32_t d_k, int32_t d_v,
                                  float scale, const void *dO, const float *dS_T, void *dq,
                                  void *dk, void *dv, float *dg, float *dbeta, float *dS0,
                                  void *workspace, size_t workspace_bytes, kda_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GDR_H */
