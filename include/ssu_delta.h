/*
 * ssu_delta.h -- the gated delta rule for speculative decode, beside the
 * selective state update of ssu.h: prompts in chunks, new tokens replayed
 * from a checkpoint through a ring, accepted tokens folded into it.
 *
 * Per value head h (key head h / (nheads_v / nheads_k)) with state
 * S [dim_v][dim_k], for every token t in order:
 *   g_t = A[h] dt',  dt' = softplus(dt_t[h] + dt_bias[h])   (or dt + dt_bias),
 *         at least -2^20 (exp is 0 from -104 on)
 *   b_t = sigmoid(beta_t[h])                                (or beta)
 *   k^ = k / sqrt(sum k^2 + 1e-6), q^ = q / sqrt(sum q^2 + 1e-6)  (or k, q)
 *   S <- exp(g_t) S;  u_t = b_t (v_t - S k^_t);  S <- S + u_t k^_t^T
 *   o_t = scale S q^_t
 * Everything between the inputs and the outputs is computed in fp32 (decay
 * sums in fp64); operands of matrix products that are not bf16 enter them in
 * three bf16 parts (24 bits) or, where the result is rounded to 16 bits anyway,
 * in two.  On ordinary inputs fp32 outputs, the final states that a prompt
 * gives beside them and fp32 checkpoints after a fold end 1e-7 to 3e-7 of their
 * norm from the exact ones; a prompt's final states beside bf16 outputs end
 * 2e-7 to 1e-6 from them, up to 4e-6 where hardly anything decays (ask for fp32
 * outputs where they have to be nearer).
 * Infinities or NaN in a token's inputs may reach every output of the call for
 * its request and head (the tokens before it in the call too), and nothing
 * else.
 *
 * The conventions of ssu.h hold: device pointers owned by the caller, nothing
 * allocated or synchronised, every kernel on the given stream of the current
 * device (calls can be captured in a HIP graph), negative codes with
 * ssu_last_error() before any launch, contract violations that only the
 * device can see skipped with a bit in *status.  Sizes of buffers are the
 * caller's: a slot id below num_slots names a page that exists, and the rows
 * that a step's cu_seqlens names are rows of its tensors (a prefill checks
 * them against `rows`).  Outputs must not overlap inputs except where it is
 * said that they may.
 */
#ifndef SSU_DELTA_H
#define SSU_DELTA_H

#include "ssu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* (entry, value head) pairs one call may cover: every launch grid, in
 * threads, then fits 32 bits.  Calls past it return SSU_ERR_UNSUPPORTED. */
#define SSU_DELTA_MAX_PAIRS (1 << 21)

/*
 * The per-slot cache.  Inside a slot page every tensor is packed; the
 * strides are BYTES between slot pages.
 *   state      [slot][nheads_v][dim_v * dim_k]     state_dtype, tiled (below)
 *   k_cache    [slot][nheads_k][ring_len][dim_k]   io_dtype (k as given, not normalised)
 *   v_cache    [slot][nheads_v][ring_len][dim_v]   io_dtype
 *   gate_cache [slot][nheads_v][ring_len][2]       f32: g_t, b_t
 *   ring_start [slot]                              i32, in [0, ring_len)
 * Live token j (j < pnat) of a slot is ring entry (ring_start + j) mod L.
 * Checkpoint tiling: rows p of dim_v in blocks of 16; value n of row
 * p = 16 rb + m, n = 16 t + 4 q + r, belongs to lane l = 16 q + m as its
 * value i = 4 t + r, and lies (e bytes a value) at byte
 *     rb * 16 * dim_k * e + (i / (16 / e) * 64 + l) * 16 + (i % (16 / e)) * e
 * (ssu_delta_init_state and ssu_delta_read_state convert from and to plain
 * row-major fp32).
 * Requirements: dim_k 64 or 128, dim_v a multiple of 16 in [16, 256],
 * nheads_v % nheads_k == 0, nheads_v * dim_v < 2^23, 1 <= ring_len <= 32,
 * state_dtype SSU_F32, SSU_BF16 or SSU_F16, io_dtype SSU_BF16; pointers 16-byte aligned (gate_cache 8-byte,
 * ring_start and status 4-byte); strides at least one packed page and
 * multiples of 16 (gate_cache: of 8).  status may be NULL.
 */
typedef struct ssu_delta_cache {
  int32_t num_slots, nheads_k, nheads_v, dim_k, dim_v, ring_len;
  ssu_dtype state_dtype;
  ssu_dtype io_dtype;
  int32_t no_qk_norm; /* nonzero: q and k are used as they are */
  void *state;
  int64_t state_slot_stride;
  void *k_cache;
  int64_t k_slot_stride;
  void *v_cache;
  int64_t v_slot_stride;
  float *gate_cache;
  int64_t gate_slot_stride;
  int32_t *ring_start;
  int32_t *status;
} ssu_delta_cache;

/*
 * One decode step, with the fields of ssu_step where they are the same.
 *   q, k  [rows][nheads_k][dim_k]  v  [rows][nheads_v][dim_v]   io_dtype,
 *         heads packed, rows q_row_stride, ... ELEMENTS apart (a multiple of
 *         8, at least one packed row)
 *   dt, beta  [rows][nheads_v] f32      A, dt_bias  [nheads_v] f32
 *   out   [rows][nheads_v][dim_v]  out_dtype (SSU_BF16 or SSU_F32)
 *   scale  the factor of q (dim_k^-1/2 in most layers)
 * Entry b's rows are b * max_seqlen + t, or [cu_seqlens[b], cu_seqlens[b+1]).
 * Requirements: 1 <= max_seqlen <= min(16, ring_len); q, k, v, out 16-byte
 * aligned, the rest 4-byte; batch * nheads_v <= SSU_DELTA_MAX_PAIRS.  Active
 * slots must be unique, in a step as in a flush and an init.  batch == 0 is a
 * no-op.
 */
typedef struct ssu_delta_step {
  int32_t batch, max_seqlen;
  const int32_t *slot_idx;
  const int32_t *prev_num_accepted;
  const int32_t *cu_seqlens;
  const void *q;
  const void *k;
  const void *v;
  int64_t q_row_stride, k_row_stride, v_row_stride;
  const float *dt;
  const float *beta;
  const float *A;
  const float *dt_bias;
  float scale;
  int32_t no_dt_softplus, no_beta_sigmoid;
  void *out;
  ssu_dtype out_dtype;
} ssu_delta_step;

/* Replays the checkpoint through the pnat live ring tokens and the entry's
 * new tokens, writes the new tokens' outputs and appends their k, v, g and b
 * to the ring.  The checkpoint and ring_start stay, so a repeated step gives
 * the same result.  Padding entries (slot <= 0 or >= num_slots) write zero
 * output rows and touch no cache; entries with pnat + T_b outside the ring
 * (SSU_STATUS_BAD_PNAT), T_b outside [0, max_seqlen] (SSU_STATUS_BAD_SEQLEN,
 * no output rows) or a bad ring_start (SSU_STATUS_BAD_RING) likewise. */
int ssu_delta_replay_step(const ssu_delta_cache *cache, const ssu_delta_step *step, hipStream_t stream);

/* Folds the first k = num_fold[j] live ring tokens of slot_idx[j] into its
 * checkpoint (fp32, rounded to nearest even once) and advances ring_start by
 * k.  k == 0 changes nothing; k outside [0, ring_len] or a bad ring_start is
 * skipped with SSU_STATUS_BAD_FOLD / SSU_STATUS_BAD_RING; padding slots are
 * ignored.  n == 0 is a no-op. */
int ssu_delta_flush(const ssu_delta_cache *cache, const int32_t *slot_idx, const int32_t *num_fold, int32_t n,
                    hipStream_t stream);

/* Writes states (f32, entry j at states + j * states_batch_stride elements,
 * [nheads_v][dim_v][dim_k] packed; stride 0 broadcasts) into the checkpoints
 * of slot_idx[j], zeroes their rings and sets ring_start to 0; ids outside
 * [1, num_slots) are ignored. */
int ssu_delta_init_state(const ssu_delta_cache *cache, const float *states, int64_t states_batch_stride,
                         const int32_t *slot_idx, int32_t n, hipStream_t stream);

/* The reverse: the checkpoints of slot_idx[j] as f32 rows (entries of ids
 * outside [1, num_slots) are left as they are). */
int ssu_delta_read_state(const ssu_delta_cache *cache, float *states, int64_t states_batch_stride,
                         const int32_t *slot_idx, int32_t n, hipStream_t stream);

/*
 * Whole sequences at once (prompts, or their next pieces).
 *   cu_seqlens [num_seqs + 1] i32: sequence s owns rows [cu[s], cu[s+1]) of
 *         the `rows` rows of q, k, v, dt, beta and out (rows behind the last
 *         sequence are left as they are).  Empty sequences are allowed.
 *   initial_states / final_states  [num_seqs][nheads_v][dim_v][dim_k] f32
 *         packed, or NULL (zero states / not wanted).  They may be the same
 *         buffer.
 *   workspace  at least ssu_delta_prefill_workspace_size() bytes, 16-byte
 *         aligned; calls that may overlap need one each.
 * q, k, v, dt, beta, A, dt_bias, out and the flags as in ssu_delta_step.  A
 * sequence whose cu_seqlens are negative, decreasing or past rows is skipped
 * and ORs SSU_STATUS_BAD_SEQLEN into *status (when not NULL); the results of
 * the call's other sequences are then not to be relied on (nothing outside
 * their rows and states is written).
 * Requirements: dim_k, dim_v and the heads as in ssu_delta_cache; rows *
 * nheads_v <= 2^30; num_seqs * nheads_v <= SSU_DELTA_MAX_PAIRS; row strides
 * below 2^23 elements.  num_seqs == 0 is a no-op; with rows == 0 the per-row tensors may be NULL.
 */
typedef struct ssu_delta_prefill_args {
  int32_t num_seqs, rows;
  int32_t nheads_k, nheads_v, dim_k, dim_v;
  ssu_dtype io_dtype;
  ssu_dtype out_dtype;
  const int32_t *cu_seqlens;
  const void *q;
  const void *k;
  const void *v;
  int64_t q_row_stride, k_row_stride, v_row_stride;
  const float *dt;
  const float *beta;
  const float *A;
  const float *dt_bias;
  float scale;
  int32_t no_dt_softplus, no_beta_sigmoid, no_qk_norm;
  const float *initial_states;
  float *final_states;
  void *out;
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;
} ssu_delta_prefill_args;

/* Bytes of scratch for `rows` rows in num_seqs sequences (0, with the reason
 * in ssu_last_error, for sizes outside the limits above). */
size_t ssu_delta_prefill_workspace_size(int32_t rows, int32_t num_seqs, int32_t nheads_v);
int ssu_delta_prefill(const ssu_delta_prefill_args *args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSU_DELTA_H */
