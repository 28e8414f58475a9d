/*
 * rsa_rows.h -- the row-local operators around Ring Self-Attention in a sequence-parallel model.
 *
 * "Sequence Parallelism: Making 4D Parallelism Possible" (Li, Xue et al., 2021; review page,
 * Abstract) splits the whole model by the sequence: only self-attention exchanges data, and
 * everything else works on a rank's own rows. rsa_sp.h has the linear layers; these are the
 * other three places where a decoder's rank works on its rows alone. The pages name none of
 * them: they are what a model on this framework needs next to its attention.
 *
 *   rsa_embed                 the rows that enter the first block, and the table's gradient
 *   rsa_qk_norm_rope          between the query/key/value projection and the attention: RMS
 *                             norm of every head's row and rotation by its position
 *   rsa_distill               behind the last projection: the loss against a teacher's top
 *                             logits (with K = 1: cross entropy), and its gradient
 *
 * Conventions as in rsa.h: plain device pointers, the current device, `stream`, nothing
 * allocated, arguments checked before anything is launched, results independent of the run
 * (no floating-point atomics). Element types RSA_BF16 and RSA_F32; statistics and sums in
 * fp32; each output rounded once, to nearest-even. Strides and leading dimensions are in
 * elements. Work on two streams must not share a workspace (nor must two captured graphs that
 * may run at the same time); a workspace needs no initial contents and keeps none between calls.
 */
#ifndef RSA_ROWS_H_
#define RSA_ROWS_H_

#include "rsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * RMS norm and rotary position of queries and keys, one pass: for every row x [d] of a head,
 *
 *   n = x * (mean(x^2) + eps)^(-1/2) * w,      y = n with its first `rot` elements rotated:
 *   (y_a, y_b) = (n_a cos t - n_b sin t, n_b cos t + n_a sin t),   t = position * freq[i]
 *
 * with the pairs (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved != 0, i < rot/2.
 * Angles are formed and reduced in fp64: off by less than 3 * 2^-53 |position * freq| + 2^-23, which is
 * less than 10^-6 while |position * freq| stays below 2^31.
 *
 * Q [B, Hq, L, d], K [B, Hk, L, d] (Hq and Hk independent) and the outputs Qo, Ko of the same
 * shapes: rows contiguous, the other strides in `strides`: (batch, head, row) of Q, K, Qo, Ko,
 * 12 numbers, each a multiple of 16 bytes (they are host memory, read during the call). So Q
 * and K may be views of the projection's output and Ko a chunk of the ring's full key buffer.
 * Qo = Q (Ko = K) with equal strides works in place; outputs that overlap an input otherwise,
 * or one another, are not allowed.
 * wq, wk: fp32 [d], or NULL for 1. freq: fp32 [rot / 2] (NULL only with rot = 0).
 * Positions: pos0 + row when pos == NULL (a rank's chunk starts at pos0 = rank * c); else
 * pos [L] (pos_batch_stride = 0) or [B, L] of int64 (pos64 != 0) or int32.
 * Supported: d in {32, 64, 128}; rot % 16 == 0, 0 <= rot <= d; B * L < 2^31; eps > 0. A row
 * whose sum of squares passes the largest fp32 number normalises to zeros, as fp32 arithmetic
 * has it. B * L == 0 launches nothing.
 */
RSA_API rsa_status_t rsa_qk_norm_rope(const void *Q, const void *K, void *Qo, void *Ko,
                                      const long long *strides, const float *wq, const float *wk,
                                      const float *freq, const void *pos, int pos64,
                                      long long pos_batch_stride, long long pos0, int B, int Hq,
                                      int Hk, int L, int d, int rot, int interleaved, float eps,
                                      rsa_dtype_t dt, void *stream);

/* Workspace bytes of rsa_qk_norm_rope_backward (the blocks' shares of the weights' gradients).
 * 0 for an unsupported d. */
RSA_API size_t rsa_qk_norm_rope_workspace_size(int d);

/*
 * Gradients of rsa_qk_norm_rope from the inputs Q, K and the outputs' gradients dQo, dKo: dQ, dK
 * (shapes of Q, K) and dwq, dwk fp32 [d] (NULL: not wanted), which are overwritten. With
 * r = (mean(x^2) + eps)^(-1/2) recomputed, dn the gradient rotated back and u = dn * w:
 *   dx = r (u - x r^2 mean(u x)),      dw = sum over B, heads, L of dn * x * r.
 * strides: (batch, head, row) of Q, K, dQo, dKo, dQ, dK: 18 numbers. dQ may be dQo or Q (dK
 * likewise) with equal strides. The rest as above. Workspace 256-byte aligned; needed only
 * when dwq or dwk is wanted. B * L == 0 writes zeros to dwq and dwk.
 */
RSA_API rsa_status_t rsa_qk_norm_rope_backward(const void *Q, const void *K, const void *dQo,
                                               const void *dKo, void *dQ, void *dK,
                                               const long long *strides, const float *wq,
                                               const float *wk, float *dwq, float *dwk,
                                               const float *freq, const void *pos, int pos64,
                                               long long pos_batch_stride, long long pos0, int B,
                                               int Hq, int Hk, int L, int d, int rot,
                                               int interleaved, float eps, rsa_dtype_t dt,
                                               void *workspace, size_t ws_bytes, void *stream);

/*
 * Embedding lookup: out[t] = scale * table[ids[t]], t < n. An id outside [0, V) gives a row of
 * zeros (padding, or another rank's part of the vocabulary).
 * ids: int64 (ids64 != 0) or int32 [n]; table [V, D] and out [n, D] of type dt, rows ld_table
 * and ld_out elements apart; no alignment beyond the element's is needed (rows on 16-byte
 * boundaries are faster). n, D >= 0 (zero launches nothing), 1 <= V < 2^31 - 1, D <= 2^20,
 * n * D < 2^40.
 */
RSA_API rsa_status_t rsa_embed(const void *ids, int ids64, const void *table, long long ld_table,
                               void *out, long long ld_out, int n, int V, int D, float scale,
                               rsa_dtype_t dt, void *stream);

/* Workspace bytes of rsa_embed_backward. 0 for invalid arguments or n * D == 0. */
RSA_API size_t rsa_embed_workspace_size(int n, int V, int D);

/*
 * The table's gradient: dtable[v] = scale * sum over t with ids[t] = v of dout[t], in the order
 * of t's within fixed pieces, so that the result does not depend on the run. Tokens are sorted
 * by id (a stable radix sort) and the sorted list is cut into pieces of equal length, so that a
 * frequent token is shared between many blocks.
 * accumulate == 0: every row of dtable [V, D] is written, zeros where no token points.
 * accumulate != 0: the sums are added to dtable (in fp32, rounded once); rows without a token
 * are neither read nor written. ids outside [0, V) have no gradient.
 * dout [n, D] of type dt; dtable of type dt_table, which is dt or RSA_F32. Alignment as above.
 * workspace: 256-byte aligned, >= rsa_embed_workspace_size(n, V, D) bytes.
 */
RSA_API rsa_status_t rsa_embed_backward(const void *ids, int ids64, const void *dout,
                                        long long ld_dout, void *dtable, long long ld_dtable,
                                        int n, int V, int D, float scale, int accumulate,
                                        rsa_dtype_t dt, rsa_dtype_t dt_table, void *workspace,
                                        size_t ws_bytes, void *stream);

/*
 * Distillation from a teacher's top logits. Row t has the student's logits z [V] and up to K
 * slots (index, teacher logit). A slot is live when its index lies in [0, V) and its teacher
 * logit is not -infinity; others are padding and nothing of them is used. With temperature tau,
 *
 *   p = softmax(teacher / tau) over the live slots,  q = softmax(z / tau) over the vocabulary,
 *   loss[t] = tau^2 sum_j p_j (ln p_j - ln q_{index_j}),     dz = dloss[t] tau (q - p).
 *
 * Slots with the same index add up. A row without a live slot has loss 0, statistics 0 and
 * gradient 0, whatever its logits. z may hold -infinity or the type's lowest value (entries not
 * in use); a row whose every logit is -infinity, or that holds a NaN, gives NaN.
 * stats[t] = (max z, ln sum exp((z - max) / tau)): what the backward pass needs.
 * In fp32 the loss is off by about 10^-6 tau^2 (1 + ln V): more than the loss itself where tau is large
 * and the live slots are nearly the whole vocabulary.
 *
 * logits [n, V], rows ld elements apart, type dt; index [n, K] int64 (index64 != 0) or int32;
 * teacher [n, K] of type teacher_dt; loss fp32 [n]; stats fp32 [n, 2] (8-byte aligned). Logits
 * need no alignment beyond the element's. 1 <= V < 2^31 - 1, 1 <= K <= RSA_DISTILL_MAX_K,
 * 1e-18 <= temperature <= 1e18, 0 <= n < 2^27 (0 launches nothing).
 */
#define RSA_DISTILL_MAX_K 1024

RSA_API rsa_status_t rsa_distill(const void *logits, long long ld, const void *index, int index64,
                                 const void *teacher, rsa_dtype_t teacher_dt, float *loss,
                                 float *stats, int n, int V, int K, float temperature,
                                 rsa_dtype_t dt, void *stream);

/* The gradient of the logits, dlogits [n, V] of type dt, rows ld_d apart (= logits with ld_d =
 * ld: in place; no other overlap), from the forward's stats and dloss: fp32, the rows'
 * gradients dloss_stride (0 or 1) elements apart. */
RSA_API rsa_status_t rsa_distill_backward(const void *logits, long long ld, const void *index,
                                          int index64, const void *teacher,
                                          rsa_dtype_t teacher_dt, const float *stats,
                                          const float *dloss, int dloss_stride, void *dlogits,
                                          long long ld_d, int n, int V, int K, float temperature,
                                          rsa_dtype_t dt, void *stream);

/* Loss and gradient in one pass, for a training loop that knows dloss beforehand (a mean's
 * 1 / n, a row weight): the logits are read from memory once. */
RSA_API rsa_status_t rsa_distill_step(const void *logits, long long ld, const void *index,
                                      int index64, const void *teacher, rsa_dtype_t teacher_dt,
                                      const float *dloss, int dloss_stride, float *loss,
                                      void *dlogits, long long ld_d, int n, int V, int K,
                                      float temperature, rsa_dtype_t dt, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RSA_ROWS_H_ */
