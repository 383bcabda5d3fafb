// Internal interface between ssu_verify (verify_api.cpp) and its kernels
// (verify_kernels.hip).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "ssu_internal.h"

namespace ssu {

enum ProbType { kPF32 = 0, kPBF16 = 1, kPF16 = 2 };

constexpr int kVerifyPiece = 1024;    // values of a row whose sum is kept: 16 a lane
constexpr int kVerifyGroup = 4096;    // of a row in one workgroup of the sums, a piece a wave
constexpr int kVerifyMaxTokens = 64;  // the drafts of an entry are tested by the lanes of one wave

inline int verify_pieces(int vocab) { return (vocab + kVerifyPiece - 1) / kVerifyPiece; }
// 8-byte words of scratch of an entry: the pieces' sums, then the verdict
inline int verify_words(int vocab) { return verify_pieces(vocab) + 2; }

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
  double *ws;                    // [batch][verify_words]
  int32_t *status;
};

hipError_t launch_verify(const KVerify &v, int prob_type, hipStream_t stream);

}  // namespace ssu
