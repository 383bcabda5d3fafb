/*
 * ssu_verify.h -- what was accepted of a step's drafted tokens: rejection
 * sampling against the target's probabilities from given uniform numbers,
 * and the ring bookkeeping that follows from it for the next call of
 * ssu.h or ssu_delta.h.
 *
 * A request b feeds T_b tokens in a step: the token emitted last, then
 * T_b - 1 drafts.  Row t of its rows holds the target's probabilities p_t
 * after token t and, for t < T_b - 1, the distribution q_t that the draft
 * d = token t + 1 came from (no draft_probs: q_t is 1 at d).
 *   d is accepted when u_t q_t(d) < p_t(d) (the product is exact) and all
 *   drafts before it were; n is the number accepted.
 *   r_i = max(p_n(i) - q_n(i), 0), rounded to fp32, when draft n + 1 was
 *   rejected, p_n(i) when there is none left; NaN counts as 0.  Where a
 *   rejected draft leaves r zero everywhere, r = p_n.
 *   The token drawn is the lowest i with r_0 + ... + r_i > u' sum r (sums in
 *   fp64), the last i with r_i > 0 if rounding leaves none.
 * Conventions as in ssu.h (device pointers, no allocation, the caller's
 * stream, graph capture, codes and ssu_last_error).
 */
#ifndef SSU_VERIFY_H
#define SSU_VERIFY_H

#include "ssu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits for ssu_verify_args.status beside those of ssu.h. */
enum {
  SSU_STATUS_BAD_TOKEN = 16, /* a drafted token outside [0, vocab): rejected, r as for no draft */
  SSU_STATUS_BAD_PROBS = 32  /* no finite positive mass to draw from: the token is -1 */
};

/*
 *   cu_seqlens  [batch + 1] i32 or NULL (row t of entry b is b * max_seqlen + t)
 *   tokens      [rows] i32, the tokens that the step was fed
 *   target_probs, draft_probs  [rows][vocab] probs_dtype (SSU_F32, SSU_BF16 or
 *               SSU_F16), rows target_row_stride / draft_row_stride ELEMENTS
 *               apart (at least vocab); draft_probs may be NULL
 *   u           [rows] f32 in [0, 1): row t's is for the draft in row t + 1
 *   u_final     [batch] f32 in [0, 1)
 *   out_tokens  [batch][max_seqlen] i32: the n accepted drafts, the drawn
 *               token, then -1
 *   num_accepted [batch] i32: n + 1, the fed tokens that stay (0 for an
 *               entry without tokens)
 * Ring bookkeeping, where next_live is not NULL: with live[b] ring tokens
 * before the step (its prev_num_accepted) of which it folded fold[b] (NULL:
 * none), next_live = live - fold + n + 1, next_fold (may be NULL) =
 * next_live where next_live + reserve > ring_len, else 0, and next_left (may
 * be NULL) = next_live - next_fold.  A flush of next_fold and a plain step
 * with prev_num_accepted = next_left need reserve = max_seqlen (also what
 * reserve 0 means); a fused step with prev_num_accepted = next_live and
 * num_fold = next_fold, which wants room for its tokens before it folds,
 * needs 2 max_seqlen.  next_live and next_left may be `live`, next_fold may
 * be `fold`.
 *   workspace   at least ssu_verify_workspace_size(batch, vocab) bytes,
 *               16-byte aligned; calls that may overlap need one each.
 * Requirements: 1 <= max_seqlen <= 64, 1 <= vocab <= 2^24, batch <= 65535,
 * batch * ceil(vocab / 4096) <= 2^23 (workgroups of a launch), the
 * probabilities aligned to their type (rows a multiple of 16 bytes apart are
 * read a little faster), the rest 4-byte.  The rows that cu_seqlens names are
 * rows of the tensors (the call does not know how many there are); a length
 * outside [0, max_seqlen] counts as none, with SSU_STATUS_BAD_SEQLEN.  An entry
 * whose residual is empty has its row read once more.  Outputs must not
 * overlap inputs except as said above.  batch == 0 is a no-op.
 */
typedef struct ssu_verify_args {
  int32_t batch, max_seqlen, vocab, ring_len, reserve;
  ssu_dtype probs_dtype;
  const int32_t *cu_seqlens;
  const int32_t *tokens;
  const void *target_probs;
  int64_t target_row_stride;
  const void *draft_probs;
  int64_t draft_row_stride;
  const float *u;
  const float *u_final;
  int32_t *out_tokens;
  int32_t *num_accepted;
  const int32_t *live;
  const int32_t *fold;
  int32_t *next_live;
  int32_t *next_fold;
  int32_t *next_left;
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;
} ssu_verify_args;

size_t ssu_verify_workspace_size(int32_t batch, int32_t vocab);
int ssu_verify(const ssu_verify_args *args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSU_VERIFY_H */
