/*
 * mimi_rvq_streams.h -- the token streams between the Mimi codec and the
 * Moshi language model, on the GPU: delay-pattern packing of the multi-stream
 * frame, its inverse, the sum of per-stream embeddings that is the Temporal
 * Transformer's input, and on the model's output side the log probabilities of
 * the streams' tokens, distillation from a teacher's top list, and gradients.
 *
 * Sources (page title, section):
 *  - "Moshi: a Speech-Text Foundation Model for Real-Time Dialogue" (notes),
 *    section 3c "Moshi - multi-stream generation": K = 17 sub-streams per
 *    12.5 Hz frame (k1 text; k2 semantic + k3..k9 acoustic of Moshi; k10
 *    semantic + k11..k17 acoustic of the user), acoustic tokens delayed by
 *    tau = 1-2 steps behind the semantic one, text before its audio.
 *  - Chinese annotated translation of the Moshi technical report: section
 *    "RQ-Transformer" (at step s the Temporal Transformer's input is the sum of
 *    K learned embedding tables of the tokens of step s - 1), "acoustic delay"
 *    and "multi-stream modeling" (the delay applies to both audio streams,
 *    which are concatenated), and the delay-pattern ablation ([0,1,...,7],
 *    [0,2,...,2], [0,0,...,0]).
 *
 * Readings (the delay equation is lost in the pages' extraction): with 0-based
 * steps, packed[s][k] = stream_k[s - delay_k] when 0 <= s - delay_k < T and the
 * stream's pad token otherwise; text and the semantic level have delay 0 (the
 * caller passes delays[0] = 0 for the standard patterns, but any delays >= 0
 * are accepted); columns are [text, stream 0 levels 0..7, stream 1 levels
 * 0..7]; pad tokens are one past each vocabulary (32000 text, 2048 audio) and
 * have their own embedding rows.
 *
 * All pointers are device pointers except where marked host; all arrays are
 * row-major and caller-owned, 16-byte aligned (the logits calls state their own
 * layout and alignment). Calls are asynchronous on
 * `stream` and allocate nothing. Status codes are those of mimi_rvq.h;
 * argument errors return at once, nothing is launched.
 */
#ifndef MIMI_RVQ_STREAMS_H
#define MIMI_RVQ_STREAMS_H

#include <stdint.h>

#include "mimi_rvq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MIMI_RVQ_TEXT_CARD 32000  /* text vocabulary (SentencePiece, 32k) */
#define MIMI_RVQ_TEXT_PAD 32000   /* pad id of the text stream */
#define MIMI_RVQ_AUDIO_PAD 2048   /* pad id of an audio stream */
#define MIMI_RVQ_MAX_STREAMS 64   /* largest K for mimi_rvq_embed_sum */
#define MIMI_RVQ_MAX_TOP 128      /* largest top_k / teacher list of the logits calls */
#define MIMI_RVQ_MAX_VOCAB (3 << 17) /* largest V of the logits calls: 393216 */

/*
 * Pack T frames into the multi-stream sequence packed [S][K], K = 1 + 8 *
 * n_audio (17 for Moshi + user). text [T] int32 (NULL: every text slot is
 * text_pad); audio [n_audio][T][8] int16 codes (n_audio 0..7); delays: host
 * [8], delays[q] >= 0 steps for level q (the same pattern for every audio
 * stream). S >= 0 steps are written (T + max delay holds every token).
 * Returns MIMI_RVQ_EINVAL on a bad argument.
 */
int mimi_rvq_delay_pack(const int32_t *text, const int16_t *audio, int n_audio, int64_t T,
                        const int32_t *delays, int64_t S, int32_t text_pad, int32_t audio_pad,
                        int32_t *packed, struct CUstream_st *stream);

/*
 * Inverse shift of one audio stream: audio [T][8] int16 with audio[t][q] =
 * packed[t + delays[q]][col0 + q], from packed [S][K] (col0 + 8 <= K, T +
 * max delay <= S, else MIMI_RVQ_EINVAL). Values are copied as they are (a pad
 * token stays 2048, which mimi_rvq_decode then reports as out of range).
 */
int mimi_rvq_delay_unpack(const int32_t *packed, int64_t S, int K, int col0,
                          const int32_t *delays, int64_t T, int16_t *audio,
                          struct CUstream_st *stream);

/*
 * out[s] = sum over k = 0..K-1 of row tokens[s][k] of table k, for s < S.
 * tables: the K tables' rows stacked, [sum rows][d], MIMI_RVQ_F32 or
 * MIMI_RVQ_BF16 (table_dtype); rows: host [K] row counts; tokens [S][K] int32;
 * out [S][d], MIMI_RVQ_F32 or MIMI_RVQ_BF16 (out_dtype). d must be a multiple
 * of 8, K in 1..MIMI_RVQ_MAX_STREAMS. The sum is taken in float32, k in order.
 * A negative token is an absent stream and adds nothing; a token >= rows[k]
 * adds nothing and is counted into *n_bad (device uint64, caller-zeroed; may
 * be NULL).
 * Failure: the bf16, d = 4096 form waits on its copies with bounded waits
 * (about 2 s). If one runs out, the kernel stops, lets the copies it issued
 * land, and returns early (the output is then undefined); it records the
 * timeout in the library's token-stream status word, which
 * mimi_rvq_streams_get_error() reports, and also sets *n_bad to UINT64_MAX
 * when n_bad is not NULL.
 */
int mimi_rvq_embed_sum(const void *tables, int table_dtype, int K, const int64_t *rows, int d,
                       const int32_t *tokens, int64_t S, void *out, int out_dtype,
                       uint64_t *n_bad, struct CUstream_st *stream);

/*
 * Status of the token-stream kernels since the last call: synchronises
 * `stream`, then returns and clears the status word that a timed-out wait of
 * mimi_rvq_embed_sum sets (MIMI_RVQ_ETIMEOUT; MIMI_RVQ_OK if none; ECUDA if a
 * CUDA call fails). The word is shared by every caller in the process.
 */
int mimi_rvq_streams_get_error(struct CUstream_st *stream);

/*
 * Failure-path self-test of mimi_rvq_embed_sum's bounded waits, without
 * hanging or faulting the GPU: launches the embedding-sum kernel in a form
 * whose producers issue no copy, so its consumers' wait runs out a short
 * budget (about 50 ms); the kernel records the timeout and returns, and the
 * next mimi_rvq_streams_get_error returns MIMI_RVQ_ETIMEOUT. Needs no buffers.
 */
int mimi_rvq_streams_wait_selftest(struct CUstream_st *stream);

/*
 * Operators on the language model's logits over the packed streams. These calls
 * share the following.
 *
 * Logits: S steps of n streams, V logits each, MIMI_RVQ_F32 or MIMI_RVQ_BF16;
 * logit i of (s, j) is element s * stride_s + j * stride_n + i (strides in
 * elements, >= 0; rows may start at any element, so the 16-byte rule does not
 * apply to logits and dlogits, nor to the other arrays of these calls, which
 * need their element's alignment). V in 1..MIMI_RVQ_MAX_VOCAB, n <= 65536. With
 * c = scale (1e-30 to 1e30; 1 / temperature):
 *     lse = ln sum_i exp(c x_i),  ln p_i = c x_i - lse,
 *     entropy = -sum_i p_i ln p_i   (0 ln 0 = 0).
 * Outputs other than dlogits are contiguous [S][n] (lists [S][n][k]) float32
 * or int32, and statistics are held in float32. S = 0 or n = 0 is a no-op.
 *
 * Tokens: the token of (s, j) is tokens[s * tok_stride_s + j * tok_stride_n]
 * (columns of packed are read where they are). A negative token and a token
 * equal to pad are no target; a token >= V other than pad is no target either
 * and is counted into *n_bad (device uint64, caller-zeroed; may be NULL).
 *
 * Special values. A logit of -inf has probability 0. A row of -inf only has no
 * distribution: lse and the logprob of a target are -inf, entropy is 0, its
 * gradient is 0. A row that holds NaN or +inf gives NaN for its values and its
 * gradient, and empty alternatives with logprob NaN. Where a row has no target
 * its logprob is 0 whatever its logits are. Logits of the type's lowest value
 * are finite: a row of nothing else is uniform. A log probability beyond
 * float32's range (such a logit times a scale above 1) is -inf, also where it
 * enters a loss.
 *
 * Gradients: dlogits has the logits' type and its own strides; its rows must
 * not share memory, and it may be the logits themselves (same pointer and
 * strides) but may not overlap them in another way (EINVAL; where the two lie
 * in each other's extent they need the same strides too). Each value is
 * computed in float32 and rounded once. A row whose upstream gradients are
 * all 0 gets zeros, whatever its logits are.
 *
 * Calls are deterministic, keep nothing between calls and may run on several
 * streams at once and be captured in CUDA graphs. Every pointer must belong to
 * the current device (or be managed memory).
 */

/*
 * Log probabilities of tokens. logprob: that of the row's token (0 without a
 * target); entropy and lse of the row; top_ids, top_logprob [S][n][top_k]: the
 * top_k most likely tokens (0..MIMI_RVQ_MAX_TOP), largest logit first, ties to
 * the lowest id; tokens of probability 0 by a logit of -inf are not listed, and
 * places left over hold id -1 and logprob -inf. Any output may be NULL; tokens
 * may be NULL when logprob is.
 */
int mimi_rvq_token_logprob(const void *logits, int dtype, int64_t S, int n, int V,
                           int64_t stride_s, int64_t stride_n, const int32_t *tokens,
                           int64_t tok_stride_s, int64_t tok_stride_n, int32_t pad, float scale,
                           int top_k, float *logprob, float *entropy, float *lse, int32_t *top_ids,
                           float *top_logprob, uint64_t *n_bad, struct CUstream_st *stream);

/*
 * Gradient of sum (g_logprob logprob + g_entropy entropy + g_lse lse) with
 * respect to the logits; g_* are [S][n] float32, NULL where there is none:
 *     dlogits_i = c (g_logprob ([i = token] - p_i) + g_lse p_i
 *                    - g_entropy p_i (ln p_i + entropy)).
 * The logits are read once and nothing of the forward call is needed. logprob,
 * entropy, lse: where not NULL, the values of mimi_rvq_token_logprob too (a
 * training step whose upstream gradients are known needs no other call).
 */
int mimi_rvq_token_logprob_grad(const void *logits, int dtype, int64_t S, int n, int V,
                                int64_t stride_s, int64_t stride_n, const int32_t *tokens,
                                int64_t tok_stride_s, int64_t tok_stride_n, int32_t pad,
                                float scale, const float *g_logprob, const float *g_entropy,
                                const float *g_lse, void *dlogits, int64_t d_stride_s,
                                int64_t d_stride_n, float *logprob, float *entropy, float *lse,
                                uint64_t *n_bad, struct CUstream_st *stream);

/*
 * Distillation from a teacher's top list: ids [S][n][k] int32 and teacher
 * [S][n][k] (MIMI_RVQ_F32 or MIMI_RVQ_BF16, teacher_dtype), k in
 * 1..MIMI_RVQ_MAX_TOP, as mimi_rvq_token_logprob writes them. An entry with a
 * negative id is empty (its value is not read into anything); an id >= V is
 * empty too and is counted into *n_bad. An id listed twice counts with both
 * entries. loss [S][n]:
 *   tail = 0: teacher holds logits or log probabilities; q = softmax(teacher)
 *             over the list, loss = sum_j q_j (ln q_j - ln p_{ids_j});
 *   tail = 1: teacher holds log probabilities t; q_j = exp(t_j), and all
 *             tokens outside the list are one more class of weight
 *             q_r = max(0, 1 - sum_j q_j) (the sum in float64) and student
 *             probability p_r: loss = sum_j q_j (t_j - ln p_{ids_j})
 *             + q_r (ln q_r - ln p_r). Where no token outside the list has
 *             probability the class is left out.
 * scale applies to the student's logits only. A term of weight 0 is 0; a list
 * without an entry (tail = 0: without weight) gives loss 0; a listed token of
 * student probability 0 by a logit of -inf gives loss +inf, and so does a row
 * of -inf only. NaN or +inf in an entry gives NaN.
 */
int mimi_rvq_distill_topk(const void *logits, int dtype, int64_t S, int n, int V, int64_t stride_s,
                          int64_t stride_n, const int32_t *ids, const void *teacher,
                          int teacher_dtype, int k, int tail, float scale, float *loss,
                          uint64_t *n_bad, struct CUstream_st *stream);

/*
 * Gradient of sum g loss with respect to the logits (g [S][n] float32; NULL:
 * all 1):
 *     dlogits_i = g c (Q p_i - sum over j with ids_j = i of q_j)  listed tokens,
 *     dlogits_i = g c (Q p_i - q_r softmax over the unlisted tokens_i)  others,
 * Q the sum of the weights (1 for tail = 0). loss: where not NULL, the losses
 * too, from the same pass.
 */
int mimi_rvq_distill_topk_grad(const void *logits, int dtype, int64_t S, int n, int V,
                               int64_t stride_s, int64_t stride_n, const int32_t *ids,
                               const void *teacher, int teacher_dtype, int k, int tail, float scale,
                               const float *g, void *dlogits, int64_t d_stride_s,
                               int64_t d_stride_n, float *loss, uint64_t *n_bad,
                               struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* MIMI_RVQ_STREAMS_H */
