// Internal interface between the host entry points of token histories and
// logits (logits_api.cpp) and their kernels (logits_kernels.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "ssu_internal.h"

namespace ssu {

constexpr int kLogitsMaxTokens = 64;  // rows of an entry
constexpr int kLogitsPiece = 2048;    // values of the smallest workgroup's piece of a row

enum LogitType { kLF32 = 0, kLBF16 = 1, kLF16 = 2 };

struct KHistory {
  int num_slots, vocab, words;
  int32_t *counts;
  int64_t counts_stride;  // i32 between pages
  uint32_t *seen;
  int64_t seen_stride;
  int32_t *status;
};

struct KCount {
  int batch, T, rows;
  const int32_t *slot_idx, *tokens, *num, *cu;
  int prompt, reset;
};

struct KLogits {
  int batch, T, rows, vocab;
  const uint8_t *in;
  int64_t in_stride;  // bytes between rows
  uint8_t *out;
  int64_t out_stride;
  const int32_t *cu, *slot_idx, *tokens;
  const float *temperature, *repetition, *frequency, *presence;
  const int32_t *bias_off, *bias_tok;
  const float *bias_val;
  int bias_count;
  const uint32_t *mask;
  int64_t mask_stride;  // words between rows
  float2 *ws;           // [batch * T][pieces]
  bool past;            // the outputs are stored past the caches
  int32_t *status;
};

// Pieces of a row that the workspace has words for.
inline int64_t logits_pieces(int64_t vocab) { return (vocab + kLogitsPiece - 1) / kLogitsPiece; }

hipError_t launch_count(const KHistory &h, const KCount &c, hipStream_t stream);
// h.counts NULL: no history
hipError_t launch_logits(const KHistory &h, const KLogits &l, int in_type, int out_type, bool softmax, hipStream_t stream);

}  // namespace ssu
