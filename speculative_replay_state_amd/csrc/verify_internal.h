// Internal interface between ssu_verify (verify_api.cpp) and its kernels
// (verify_kernels.hip).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "ssu_internal.h"

namespace ssu {

enum ProbType { kPF32 = 0, kPBF16 = 1, kPF16 = 2 };

constexpr int kVerifySeg = 4096;      // values of a row per workgroup of the first kernel
constexpr int kVerifyMaxTokens = 64;  // the drafts of an entry are tested by the lanes of one wave

inline int verify_segments(int vocab) { return (vocab + kVerifySeg - 1) / kVerifySeg; }

struct KVerify {
  int batch, T, vocab, ring_len, reserve;
  const int32_t *cu;
  const int32_t *tokens;
  const uint8_t *p, *q;          // q: NULL without draft probabilities
  int64_t p_stride, q_stride;    // bytes between rows
  const float *u, *uf;
  int32_t *out, *accepted;
  const int32_t *live, *fold;
  int32_t *next_live, *next_fold, *next_left;
  double *ws;                    // [batch][segments]
  int32_t *status;
  int wide;                      // rows can be read 16 bytes at a time
};

hipError_t launch_verify(const KVerify &v, int prob_type, hipStream_t stream);

}  // namespace ssu
