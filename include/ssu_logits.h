/*
 * ssu_logits.h -- from a step's logits to the probabilities that ssu_verify
 * takes: penalties for repeated tokens, biases, grammar masks, temperature and
 * softmax, and the counts of a request's tokens that the penalties go by.
 *
 * A loop of a request then is ssu_history_count of its prompt (reset, prompt),
 * and for every step: ssu_logits, ssu_verify, ssu_history_count of what that
 * emitted (out_tokens, num_accepted as they are).  Conventions as in ssu.h
 * (device pointers, no allocation, the caller's stream, graph capture, codes
 * and ssu_last_error).
 */
#ifndef SSU_LOGITS_H
#define SSU_LOGITS_H

#include "ssu_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits for the status words here, beside those of ssu.h and ssu_verify.h. */
enum {
  SSU_STATUS_EMPTY_ROW = 64, /* nothing of a row can be taken: its probabilities are 0 */
  SSU_STATUS_BAD_BIAS = 128  /* bias_offsets outside [0, bias_count] or decreasing (the entry then
                                has no biases), or a biased token outside [0, vocab) (not applied) */
};

/*
 * The tokens of the requests in num_slots cache slots.
 *   counts [slot][vocab] i32: 2 n + p, n times generated, p = 1 if the prompt
 *          holds the token; a word counts where its bit in `seen` is set and
 *          holds anything elsewhere
 *   seen   [slot][ceil(vocab / 32)] u32: bit i % 32 of word i / 32 is set for
 *          every token i that the request holds
 * Strides are BYTES between slot pages, multiples of 4 and at least one packed
 * page.  A slot's page begins with a count whose reset is set; slots as in
 * ssu.h (slot 0 is the padding slot).  status: NULL or a word that the count and the
 * logits OR bits into.  1 <= vocab <= 2^24; pointers 4-byte aligned.
 */
typedef struct ssu_history {
  int32_t num_slots, vocab;
  int32_t *counts;
  int64_t counts_slot_stride;
  uint32_t *seen;
  int64_t seen_slot_stride;
  int32_t *status;
} ssu_history;

/*
 * Tokens counted in the pages of slot_idx [batch] (ids outside [1, num_slots)
 * are ignored; active slots must be unique).
 *   tokens      [rows] i32.  cu_seqlens [batch + 1] i32: entry b's are
 *               [cu_seqlens[b], cu_seqlens[b + 1]).  NULL: they begin at b *
 *               max_seqlen, and are num_tokens[b] (NULL: max_seqlen), as
 *               ssu_verify leaves its out_tokens and num_accepted.
 *   prompt      nonzero: the tokens are the prompt's (p); 0: generated (n + 1
 *               for each).
 *   reset       nonzero: the page is emptied first.
 * A token outside [0, vocab) is left out (SSU_STATUS_BAD_TOKEN); an entry whose
 * number is outside [0, max_seqlen], or whose cu_seqlens are negative,
 * decreasing or past rows, is skipped (SSU_STATUS_BAD_SEQLEN), its page left
 * as it is.  Requirements: batch <= 2^20, rows <= 2^30, max_seqlen >= 1
 * without cu_seqlens (ignored with them), rows >= batch * max_seqlen then;
 * pointers 4-byte aligned.  batch == 0 is a no-op; with rows == 0 tokens may be NULL.
 */
typedef struct ssu_count_args {
  int32_t batch, max_seqlen, rows;
  const int32_t *slot_idx;
  const int32_t *tokens;
  const int32_t *num_tokens;
  const int32_t *cu_seqlens;
  int32_t prompt, reset;
} ssu_count_args;

int ssu_history_count(const ssu_history *history, const ssu_count_args *args, hipStream_t stream);

/*
 * The logits of a step's rows, entry b's in rows b * max_seqlen + t or
 * [cu_seqlens[b], cu_seqlens[b + 1]) as in ssu_step.  For row t of entry b and
 * token i, in fp32, every operation rounded:
 *   x = l_i + bias_b(i)                           (where i has one)
 *   where i is in the history of slot_idx[b] or among the entry's tokens
 *   1 .. t (the drafts fed up to this row; token 0 was emitted before and is
 *   in the history):
 *     x = x > 0 ? x / repetition[b] : x * repetition[b]
 *     x = x - (frequency[b] n + (n > 0 ? presence[b] : 0)),  n = times
 *     generated plus times among those drafts
 *   where the row's mask bit of i is 0, or x is NaN: the token is left out (x
 *   = -inf)
 *   p_i = exp(x_i / temperature[b]) / sum,  rounded to out_dtype
 * temperature <= 0 (or NaN): p = 1 at the lowest i of the largest x.  In both x
 * = +inf counts as the largest finite value.  A row with no x above -inf is
 * all 0 and ORs SSU_STATUS_EMPTY_ROW.  With no_softmax the outputs are x /
 * temperature (x itself where that is <= 0 or NaN; -inf stays -inf), rounded to
 * out_dtype, and nothing is said of empty rows.
 *
 *   logits, out  [rows][vocab], logits_dtype / out_dtype (SSU_F32, SSU_BF16 or
 *                SSU_F16), rows *_row_stride ELEMENTS apart (at least vocab),
 *                aligned to their type.  out may be logits itself (same type and
 *                stride).
 *   temperature, repetition, frequency, presence  [batch] f32 or NULL (1, 1, 0, 0)
 *   slot_idx     [batch] i32, the history's slots (ids outside [1, num_slots):
 *                an empty history); may be NULL without a history
 *   tokens       [rows] i32, what the step was fed, or NULL: no drafts are
 *                counted.  A draft outside [0, vocab) is not counted.
 *   bias_offsets [batch + 1] i32, bias_tokens, bias_values [bias_count]: entry
 *                b's biases are [bias_offsets[b], bias_offsets[b + 1]), in any
 *                order; of a token that comes more than once the last one
 *                holds.  NULL: none.
 *   mask         [rows][ceil(vocab / 32)] u32, mask_row_stride WORDS apart (0: one
 *                mask for all rows): bit i % 32 of word i / 32 set where token
 *                i may be taken.  NULL: all.
 *   workspace    at least ssu_logits_workspace_size() bytes, 16-byte aligned;
 *                calls that may overlap need one each.  NULL with no_softmax.
 * history NULL: tokens (and slot_idx) are not read, and repetition, frequency and
 * presence must be NULL.  Rows that no entry owns are left as they are, and an
 * entry whose length is outside [0, max_seqlen], or whose cu_seqlens are negative,
 * decreasing or past rows, is skipped (SSU_STATUS_BAD_SEQLEN).
 * Requirements: 1 <= max_seqlen <= 64, 1 <= vocab <= 2^24 (the history's too),
 * batch * max_seqlen <= 65535, batch * max_seqlen * ceil(vocab / 2048) <= 2^23
 * (workgroups of a launch), bias_count < 2^24, rows >= batch * max_seqlen without cu_seqlens, the
 * index and parameter arrays and the mask 4-byte aligned.  batch == 0 is a no-op.
 */
typedef struct ssu_logits_args {
  int32_t batch, max_seqlen, rows, vocab;
  ssu_dtype logits_dtype, out_dtype;
  const void *logits;
  int64_t logits_row_stride;
  void *out;
  int64_t out_row_stride;
  const int32_t *cu_seqlens;
  const int32_t *slot_idx;
  const int32_t *tokens;
  const float *temperature, *repetition, *frequency, *presence;
  const int32_t *bias_offsets;
  const int32_t *bias_tokens;
  const float *bias_values;
  int32_t bias_count;
  const uint32_t *mask;
  int64_t mask_row_stride;
  int32_t no_softmax;
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;
} ssu_logits_args;

/* Bytes of scratch for batch entries of up to max_seqlen rows (0, with the
 * reason in ssu_last_error, for sizes outside the limits above). */
size_t ssu_logits_workspace_size(int32_t batch, int32_t max_seqlen, int32_t vocab);
int ssu_logits(const ssu_history *history, const ssu_logits_args *args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSU_LOGITS_H */
