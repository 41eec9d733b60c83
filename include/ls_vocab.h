/*
 * ls_vocab.h -- C ABI of the vocabulary operators for NVIDIA GB300 (sm_103a),
 * libls_vocab.so: what a language model's training step and its scoring run
 * where hidden states meet the vocabulary.  They stand next to the criterion
 * and the embedding of ls_ops.h:
 *  - linear cross entropy: the output projection fused with its softmax cross
 *    entropy and with its gradient, in pieces of the vocabulary, so that the
 *    logits are never kept;
 *  - distillation from a teacher's top logits, forward and backward;
 *  - embedding lookup with scaling, and its gradient summed by sorted tokens.
 *
 * Conventions are those of ls_ops.h (status codes, storage types with FP32
 * arithmetic, row-major contiguous 16-byte aligned device buffers owned by
 * the caller, nothing allocated, nothing synchronised, all work enqueued on
 * `stream`, argument errors returned before anything is enqueued), and:
 *  - Storage may also be BF16 (LS_BF16).
 *  - int32 arrays (targets, tokens, teacher indices) and FP32 per-row arrays
 *    need 4-byte alignment only, teacher logits that of their element.
 *  - No output may overlap an input, another output or the workspace, except
 *    where an entry point says so.
 *  - A workspace is scratch: it needs no initialisation and holds nothing
 *    between calls, so calls ordered on one stream (or graphs whose replays
 *    are ordered) may share one.  Calls that can run at the same time on the
 *    GPU must not; nor may a workspace that a reduction of ls_ops.h still
 *    reads on its second stream (ls_set_reduction_stream) be given to these
 *    calls before ls_join_reductions: they do not know of it.
 *  - Results do not depend on the run: every sum is added in an order that
 *    the shapes and the ids fix, without floating-point atomics.
 */
#ifndef LS_VOCAB_H
#define LS_VOCAB_H

#include <stddef.h>
#include <stdint.h>

#include "ls_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Message of this library's last failing call on this host thread ("" if none). */
const char* ls_vocab_last_error(void);

/* ls_check_device_errors for this library's kernels: waits for all work on
 * the current device, returns the OR of the failure flags raised since the
 * previous call (LS_DEVERR_WAIT_TIMEOUT: a bounded wait for a bulk copy or a
 * tensor-core product ran out, and that call's outputs are incomplete) and
 * clears them. */
ls_status ls_vocab_check_device_errors(uint32_t* flags);

/* Self-test of that failure path, as ls_selftest_wait_timeout: enqueues two
 * warps that wait on a barrier which nothing completes, for `polls` polls
 * (1 .. 2^19, each up to about 2 us); LS_DEVERR_WAIT_TIMEOUT is recorded and
 * they exit. */
ls_status ls_vocab_selftest_wait_timeout(uint32_t polls, void* stream);

/* Linear cross entropy.  x: [rows, hidden], weight: [vocab, hidden], both in
 * the storage dtype (LS_F16 or LS_BF16), target: int32 [rows].  With
 *   z[i,j]  = sum_c x[i,c] * weight[j,c]          (products and sums in FP32, never rounded to 16 bits)
 *   lse[i]  = log sum_j exp(z[i,j])
 *   loss[i] = (1 - eps) * (lse[i] - z[i,target]) + eps * (lse[i] - mean_j z[i,j])
 * as ls_cross_entropy_fwd computes them from given logits.  hidden must be a
 * multiple of 8 and at most 65536; any vocab from 1 to 2^30, any rows up to
 * 2^24, as long as rows * vocab is at most 2^46 and vocab * hidden 2^40.  A target equal to ignore_index, or outside [0, vocab), gives loss 0;
 * its lse is still written.  loss and lse: FP32 [rows]; lse may be NULL.
 * workspace: at least ls_linear_cross_entropy_fwd_workspace_bytes bytes. */
ls_status ls_linear_cross_entropy_fwd(ls_dtype dtype, float* loss, float* lse, const void* x,
                                      const void* weight, const int32_t* target, int64_t rows,
                                      int64_t hidden, int64_t vocab, float label_smoothing,
                                      int32_t ignore_index, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* Backward of the above, from the forward's lse.  The logits are computed
 * again, one piece of the vocabulary at a time, and
 *   g[i,j]       = dloss[i] * (exp(z[i,j] - lse[i]) - (1 - eps) * [j == target[i]] - eps / vocab)
 *   dx[i,c]      = sum_j g[i,j] * weight[j,c]
 *   dweight[j,c] = sum_i g[i,j] * x[i,c]
 * g is rounded once to the storage dtype for the two products, after a
 * division by max|dloss| (1 - eps) which the FP32 sums undo (FP16 keeps
 * values down to 2^-38 of the largest dloss that way).  The sums run in the
 * tensor cores' accumulators, which drop low bits, over at most 16384 rows or
 * 32768 entries (9e-5 and 2e-4 of a sum of terms of one sign), and in FP32
 * from there on.
 * dloss: FP32 [rows] or NULL for 1.  Rows with an ignored target contribute
 * nothing and get a zero dx, whatever they and their dloss hold (NaN too).
 * dx: [rows, hidden] in the storage dtype, written, or NULL.
 * dweight: [vocab, hidden], or NULL; with dweight_dtype == dtype it is
 * written; with dweight_dtype == LS_F32 the gradient is ADDED to it, as
 * ls_embedding_bwd and ls_embedding_lookup_bwd add to theirs, so that tied
 * embeddings share one gradient.  rows == 0 writes zeros to a dweight in the
 * storage dtype.
 * workspace: at least ls_linear_cross_entropy_workspace_bytes bytes. */
ls_status ls_linear_cross_entropy_bwd(ls_dtype dtype, void* dx, void* dweight,
                                      ls_dtype dweight_dtype, const void* x, const void* weight,
                                      const int32_t* target, const float* lse, const float* dloss,
                                      int64_t rows, int64_t hidden, int64_t vocab,
                                      float label_smoothing, int32_t ignore_index,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes that either call above can do with for these sizes: for the
 * backward, a piece of the vocabulary's gradients (128 MB or 2048 columns of
 * them at the most), a copy of x, up to 16 FP32 copies of dx and, beyond 16384
 * rows, a piece of dweight in FP32.  0 for invalid sizes. */
size_t ls_linear_cross_entropy_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab);

/* What the forward alone needs, as a program that only scores does: 24 bytes
 * for each row and 256 (or fewer) columns. */
size_t ls_linear_cross_entropy_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab);

/* Distillation from a teacher's top logits.  logits: [rows, vocab] of the
 * student (LS_F32, LS_F16 or LS_BF16; vocab a multiple of 8), teacher_index:
 * int32 [rows, k] and teacher_logits: [rows, k] in the same storage dtype, the
 * k vocabulary entries that the teacher gave for the row, in any order.  With
 * temperature tau, 2^-60 to 2^60, and, for the valid entries e (index in [0, vocab)),
 *   log q[e] = t[e] / tau - teacher_lse[row]     or, with teacher_lse == NULL,
 *   log q[e] = t[e] / tau - log sum_valid exp(t / tau)     (renormalised over the entries)
 *   log p[j] = z[j] / tau - lse[row],  lse[row] = log sum_j exp(z[j] / tau)
 *   loss[row] = tau^2 * sum_e q[e] * (log q[e] - log p[index[e]])
 * teacher_lse (FP32 [rows]) is the log-sum-exp of the teacher's whole row of
 * t / tau: the entries then keep their true probabilities, whose sum is below
 * 1, and the teacher's tail is left out.  An entry with a logit of -inf, or
 * an index outside [0, vocab) (such as -1, for a row with fewer entries), has
 * q = 0 and adds nothing; a row without entries has loss 0.  An index that a
 * row holds twice counts twice.  1 <= k <= 1024.  loss and lse: FP32 [rows],
 * lse may be NULL.  Masks may be -inf or any finite value: a row of nothing
 * but one has the lse that FP32 can hold, the mask / tau itself where
 * log(vocab) is below its last place. */
ls_status ls_distill_topk_fwd(ls_dtype dtype, float* loss, float* lse, const void* logits,
                              const int32_t* teacher_index, const void* teacher_logits,
                              const float* teacher_lse, int64_t rows, int64_t vocab, int64_t k,
                              float temperature, void* stream);

/* Backward of the above, from the forward's lse:
 *   dlogits[j] = dloss[row] * tau * (p[j] * sum_e q[e] - sum_{e: index[e] == j} q[e])
 * dloss: FP32 [rows], or NULL for 1.  A row whose q are all 0 gets a zero
 * gradient.  dlogits may be logits (in place).  p carries the rounding of the
 * FP32 lse, |lse| * 2^-24 relative; it is at most 1 wherever lse is the
 * forward's. */
ls_status ls_distill_topk_bwd(ls_dtype dtype, void* dlogits, const void* logits,
                              const int32_t* teacher_index, const void* teacher_logits,
                              const float* lse, const float* teacher_lse, const float* dloss,
                              int64_t rows, int64_t vocab, int64_t k, float temperature,
                              void* stream);

/* Embedding lookup with scaling.  tokens: int32 [tokens_count], table:
 * [vocab, hidden] (LS_F32, LS_F16 or LS_BF16; hidden a multiple of 8):
 *   y[i] = scale * table[tokens[i]]     (FP32 product, rounded once)
 * An id outside [0, vocab) gives a zero row. */
ls_status ls_embedding_lookup_fwd(ls_dtype dtype, void* y, const int32_t* tokens,
                                  const void* table, int64_t tokens_count, int64_t hidden,
                                  int64_t vocab, float scale, void* stream);

/* Gradient of the table, FP32 [vocab, hidden]:
 *   d_table[w] = scale * sum over tokens i with id w of dy[i]     (dy in the storage dtype)
 * accumulate == 0: d_table is written whole, zeros for ids that no token has;
 * accumulate != 0: the sums are added to it.  Tokens equal to padding_id, or
 * outside [0, vocab), add nothing (padding_id outside the table: none).
 * Unlike ls_embedding_bwd the cost grows with the tokens, not with their
 * square: the tokens are sorted by id (stably), and each id's rows are added
 * in token order, in runs of a fixed length whose sums are then added in
 * order.  tokens_count up to 2^30; vocab up to 2^30.  workspace: at least
 * ls_embedding_lookup_workspace_bytes bytes. */
ls_status ls_embedding_lookup_bwd(ls_dtype dtype, float* d_table, const void* dy,
                                  const int32_t* tokens, int64_t tokens_count, int64_t hidden,
                                  int64_t vocab, float scale, int32_t padding_id, int accumulate,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of ls_embedding_lookup_bwd for these sizes; 0 for invalid sizes. */
size_t ls_embedding_lookup_workspace_bytes(int64_t tokens_count, int64_t hidden, int64_t vocab);

#ifdef __cplusplus
}
#endif
#endif /* LS_VOCAB_H */
