/*
 * ssu_prefill.h -- whole sequences (prompts, or their next pieces) under the
 * selective state update of ssu.h, and the way back from a cache slot's
 * checkpoint to fp32 states: what comes before ssu_init_state and after a
 * request's last flush.
 *
 * Per head h (group h / (nheads / ngroups)) with state S [64][128], for every
 * token t of a sequence in order:
 *   dt' = softplus(dt_t[h] + dt_bias[h])                  (or dt + dt_bias)
 *   S <- exp(A[h] dt') S + dt' x_t B_t^T
 *   y_t = S C_t + D[h] x_t,  out_t = y_t  or  y_t z_t sigmoid(z_t)
 * A[h] dt' is at least -2^20 (exp is 0 from -104 on).  Everything between the
 * inputs and the outputs is computed in fp32 (decay sums in fp64); operands of
 * matrix products that are not bf16 enter them in three bf16 parts (24 bits).
 * bf16 outputs are the fp32 ones rounded once.  Infinities or NaN in a token's
 * inputs may reach every output of the call for its sequence and head (from B
 * and C: of the heads of its group), the tokens before it too, and nothing else.
 *
 * The conventions of ssu.h hold: device pointers owned by the caller, nothing
 * allocated or synchronised, every kernel on the given stream of the current
 * device (calls can be captured in a HIP graph), negative codes with
 * ssu_last_error() before any launch, contract violations that only the
 * device can see skipped with a bit in *status.  Outputs must not overlap
 * inputs except where it is said that they may.
 */
#ifndef SSU_PREFILL_H
#define SSU_PREFILL_H

#include "ssu.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   cu_seqlens [num_seqs + 1] i32: sequence s owns rows [cu[s], cu[s+1]) of
 *         the `rows` rows of x, B, C, dt, z and out (rows behind the last
 *         sequence are left as they are).  Empty sequences are allowed.
 *   x, z  [rows][nheads][64]  B, C  [rows][ngroups][128]   io_dtype, heads and
 *         groups packed, rows x_row_stride, ... ELEMENTS apart (a multiple of
 *         8, at least one packed row: slices of a projection's rows).  z may be
 *         NULL: no gate.
 *   dt    [rows][nheads] f32       A, D, dt_bias  [nheads] f32
 *   out   [rows][nheads][64]       out_dtype (SSU_BF16 or SSU_F32), packed
 *   initial_states / final_states  [num_seqs][nheads][64][128] f32 packed (as
 *         ssu_init_state takes and ssu_read_state gives them), or NULL (zero
 *         states / not wanted).  They may be the same buffer.
 *   workspace  at least ssu_prefill_workspace_size() bytes, 16-byte aligned;
 *         calls that may overlap need one each.
 *   status  NULL, or a word that bits are ORed into.
 * A sequence whose cu_seqlens are negative, decreasing or past rows is skipped
 * and ORs SSU_STATUS_BAD_SEQLEN into *status; the results of the call's other
 * sequences are then not to be relied on (nothing outside their rows and states
 * is written).
 * Requirements: headdim == 64, dstate == 128, nheads % ngroups == 0, io_dtype
 * SSU_BF16; nheads <= 32768; rows * nheads <= 2^30; num_seqs * nheads <=
 * 2^20; row strides below 2^23 elements; x, B, C, z, out, states and workspace
 * 16-byte aligned, the rest 4-byte.  num_seqs == 0 is a no-op; with rows == 0
 * the per-row tensors may be NULL.
 */
typedef struct ssu_prefill_args {
  int32_t num_seqs, rows;
  int32_t nheads, ngroups, headdim, dstate;
  ssu_dtype io_dtype;
  ssu_dtype out_dtype;
  const int32_t *cu_seqlens;
  const void *x;
  const void *B;
  const void *C;
  const void *z;
  int64_t x_row_stride, B_row_stride, C_row_stride, z_row_stride;
  const float *dt;
  const float *A;
  const float *D;
  const float *dt_bias;
  int32_t no_dt_softplus;
  const float *initial_states;
  float *final_states;
  void *out;
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;
} ssu_prefill_args;

/* Bytes of scratch for `rows` rows in num_seqs sequences, whatever their
 * lengths; it is enough for fewer of both (0, with the reason in ssu_last_error,
 * for sizes outside the limits above). */
size_t ssu_prefill_workspace_size(int32_t rows, int32_t num_seqs, int32_t nheads);
int ssu_prefill(const ssu_prefill_args *args, hipStream_t stream);

/*
 * The reverse of ssu_init_state: the checkpoints of slot_idx[j] as fp32 states
 * at states + j * states_batch_stride elements, [nheads][64][128] packed.
 * recur == 0 reads `state`, the checkpoint that steps read; nonzero reads
 * recur_state (SSU_ERR_INVALID where the cache has none).  Values are decoded
 * exactly but for one rounding to fp32 (fp8: code * scale; nvfp4: code * block
 * scale, which is exact, times the slot's scale); the tokens of the ring are not folded in
 * (flush them first).  Entries of ids outside [1, num_slots) are left as they
 * are; an id may come more than once.  n == 0 is a no-op, n < 0
 * SSU_ERR_INVALID, n * nheads > 2^21 SSU_ERR_UNSUPPORTED; states 16-byte
 * aligned, states_batch_stride a multiple of 4 and at least one packed state;
 * slot_idx 4-byte aligned.
 */
int ssu_read_state(const ssu_cache *cache, float *states, int64_t states_batch_stride, const int32_t *slot_idx, int32_t n,
                   int32_t recur, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSU_PREFILL_H */
