// Host entry points of include/ssu_verify.h: argument checks and the launch.
#include <cstring>

#include <hip/hip_runtime.h>

#include "../../include/ssu_verify.h"
#include "verify_internal.h"

namespace {

using ssu::api_fail;
using ssu::api_ok;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_sizes(int32_t batch, int32_t vocab) {
  if (batch < 0) return api_fail(SSU_ERR_INVALID, "batch must be >= 0 (got %d)", batch);
  if (batch > 65535) return api_fail(SSU_ERR_UNSUPPORTED, "batch %d exceeds 65535 entries per call", batch);
  if (vocab < 1) return api_fail(SSU_ERR_INVALID, "vocab must be positive (got %d)", vocab);
  if (vocab > (1 << 24)) return api_fail(SSU_ERR_UNSUPPORTED, "vocab %d exceeds 2^24", vocab);
  if ((int64_t)batch * ((vocab + ssu::kVerifyGroup - 1) / ssu::kVerifyGroup) > (1 << 23))  // a grid's threads fit 32 bits
    return api_fail(SSU_ERR_UNSUPPORTED, "batch %d x vocab %d exceeds 2^23 workgroups of %d values per call", batch, vocab,
                    ssu::kVerifyGroup);
  return SSU_OK;
}

size_t bytes_for(int64_t batch, int32_t vocab) { return (size_t)(batch * ssu::verify_words(vocab)) * sizeof(double); }

}  // namespace

extern "C" {

size_t ssu_verify_workspace_size(int32_t batch, int32_t vocab) {
  if (check_sizes(batch, vocab) != SSU_OK) return 0;
  api_ok();
  return bytes_for(batch, vocab);
}

int ssu_verify(const ssu_verify_args *a, hipStream_t stream) {
  if (!a) return api_fail(SSU_ERR_INVALID, "verify descriptor is NULL");
  const int rc = check_sizes(a->batch, a->vocab);
  if (rc != SSU_OK) return rc;
  if (a->max_seqlen < 1) return api_fail(SSU_ERR_INVALID, "max_seqlen must be >= 1 (got %d)", a->max_seqlen);
  if (a->max_seqlen > ssu::kVerifyMaxTokens)
    return api_fail(SSU_ERR_UNSUPPORTED, "max_seqlen %d exceeds %d", a->max_seqlen, ssu::kVerifyMaxTokens);
  int32_t pt;
  std::memcpy(&pt, &a->probs_dtype, sizeof pt);
  if (pt != SSU_F32 && pt != SSU_BF16 && pt != SSU_F16)
    return api_fail(SSU_ERR_UNSUPPORTED, "probs_dtype must be SSU_F32, SSU_BF16 or SSU_F16 (got %d)", pt);
  const int64_t size = pt == SSU_F32 ? 4 : 2;
  if (a->batch == 0) return api_ok();
  if (!a->tokens || !a->target_probs || !a->u || !a->u_final || !a->out_tokens || !a->num_accepted)
    return api_fail(SSU_ERR_INVALID, "tokens, target_probs, u, u_final, out_tokens and num_accepted must not be NULL");
  if (a->target_row_stride < a->vocab || (a->draft_probs && a->draft_row_stride < a->vocab))
    return api_fail(SSU_ERR_INVALID, "the row strides of the probabilities must be at least vocab (%d)", a->vocab);
  if (!aligned(a->target_probs, size) || !aligned(a->draft_probs, size))
    return api_fail(SSU_ERR_INVALID, "the probabilities must be aligned to their type");
  if (!aligned(a->cu_seqlens, 4) || !aligned(a->tokens, 4) || !aligned(a->u, 4) || !aligned(a->u_final, 4) ||
      !aligned(a->out_tokens, 4) || !aligned(a->num_accepted, 4) || !aligned(a->live, 4) || !aligned(a->fold, 4) ||
      !aligned(a->next_live, 4) || !aligned(a->next_fold, 4) || !aligned(a->next_left, 4) || !aligned(a->status, 4))
    return api_fail(SSU_ERR_INVALID, "the index, number and status arrays must be 4-byte aligned");
  if (a->next_live) {
    if (!a->live) return api_fail(SSU_ERR_INVALID, "next_live needs live");
    if (a->reserve < 0) return api_fail(SSU_ERR_INVALID, "reserve must be >= 0 (got %d)", a->reserve);
    if (a->ring_len < a->max_seqlen || a->ring_len < a->reserve)
      return api_fail(SSU_ERR_INVALID, "ring_len %d is smaller than max_seqlen %d or reserve %d", a->ring_len, a->max_seqlen,
                      a->reserve);
  } else if (a->next_fold || a->next_left) {
    return api_fail(SSU_ERR_INVALID, "next_fold and next_left need next_live");
  }
  const size_t need = bytes_for(a->batch, a->vocab);
  if (!a->workspace || a->workspace_bytes < need)
    return api_fail(SSU_ERR_WORKSPACE, "verification needs a workspace of %zu bytes (got %zu%s)", need, a->workspace_bytes,
                    a->workspace ? "" : ", NULL");
  if (!aligned(a->workspace, 16)) return api_fail(SSU_ERR_INVALID, "workspace must be 16-byte aligned");
  ssu::KVerify v;
  v.batch = a->batch;
  v.T = a->max_seqlen;
  v.vocab = a->vocab;
  v.ring_len = a->ring_len;
  v.reserve = a->reserve ? a->reserve : a->max_seqlen;
  v.cu = a->cu_seqlens;
  v.tokens = a->tokens;
  v.p = static_cast<const uint8_t *>(a->target_probs);
  v.q = static_cast<const uint8_t *>(a->draft_probs);
  v.p_stride = a->target_row_stride * size;
  v.q_stride = a->draft_row_stride * size;
  v.u = a->u;
  v.uf = a->u_final;
  v.out = a->out_tokens;
  v.accepted = a->num_accepted;
  v.live = a->live;
  v.fold = a->fold;
  v.next_live = a->next_live;
  v.next_fold = a->next_fold;
  v.next_left = a->next_left;
  v.ws = static_cast<double *>(a->workspace);
  v.status = a->status;
  const hipError_t err = ssu::launch_verify(v, pt == SSU_F32 ? ssu::kPF32 : (pt == SSU_BF16 ? ssu::kPBF16 : ssu::kPF16), stream);
  return err == hipSuccess ? api_ok() : api_fail(SSU_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(err));
}

}  // extern "C"
