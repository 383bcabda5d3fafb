// Host entry points of token histories and logits (include/ssu_logits.h):
// argument checks and launches.
#include <cstring>

#include <hip/hip_runtime.h>

#include "../../include/ssu_logits.h"
#include "logits_internal.h"

namespace {

using ssu::api_fail;
using ssu::api_ok;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// An enum field as its 32 bits: a C caller may store any int.
template <class E>
int32_t raw(const E &e) {
  static_assert(sizeof(E) == sizeof(int32_t), "the ABI's enums are 32-bit");
  int32_t v;
  std::memcpy(&v, &e, sizeof v);
  return v;
}

int logit_type(int32_t t) {
  return t == SSU_F32 ? ssu::kLF32 : t == SSU_BF16 ? ssu::kLBF16 : t == SSU_F16 ? ssu::kLF16 : -1;
}

constexpr int32_t kMaxCountRows = 1 << 30;  // an index steps past an entry's last token by up to 4096

int check_vocab(int32_t vocab) {
  if (vocab < 1) return api_fail(SSU_ERR_INVALID, "vocab must be positive (got %d)", vocab);
  if (vocab > (1 << 24)) return api_fail(SSU_ERR_UNSUPPORTED, "vocab %d exceeds 2^24", vocab);
  return SSU_OK;
}

int check_history(const ssu_history *h) {
  if (h->num_slots < 1) return api_fail(SSU_ERR_INVALID, "num_slots must be positive (got %d)", h->num_slots);
  const int rc = check_vocab(h->vocab);
  if (rc != SSU_OK) return rc;
  if (!h->counts || !h->seen) return api_fail(SSU_ERR_INVALID, "counts and seen must not be NULL");
  if (!aligned(h->counts, 4) || !aligned(h->seen, 4) || !aligned(h->status, 4))
    return api_fail(SSU_ERR_INVALID, "counts, seen and status must be 4-byte aligned");
  const struct {
    const char *name;
    int64_t stride, need;
  } s[] = {{"counts", h->counts_slot_stride, (int64_t)h->vocab * 4}, {"seen", h->seen_slot_stride, ((int64_t)h->vocab + 31) / 32 * 4}};
  for (const auto &t : s) {
    if (t.stride < t.need)
      return api_fail(SSU_ERR_INVALID, "%s slot stride %lld is smaller than one packed slot (%lld bytes)", t.name,
                      (long long)t.stride, (long long)t.need);
    if (t.stride % 4 != 0)
      return api_fail(SSU_ERR_INVALID, "%s slot stride %lld is not a multiple of 4 bytes", t.name, (long long)t.stride);
  }
  return SSU_OK;
}

ssu::KHistory khistory(const ssu_history *h) {
  ssu::KHistory k;
  std::memset(&k, 0, sizeof k);
  if (!h) return k;
  k.num_slots = h->num_slots;
  k.vocab = h->vocab;
  k.words = (h->vocab + 31) / 32;
  k.counts = h->counts;
  k.counts_stride = h->counts_slot_stride / 4;
  k.seen = h->seen;
  k.seen_stride = h->seen_slot_stride / 4;
  k.status = h->status;
  return k;
}

int check_sizes(int32_t batch, int32_t T, int32_t vocab) {
  if (batch < 0) return api_fail(SSU_ERR_INVALID, "batch must be >= 0 (got %d)", batch);
  if (T < 1) return api_fail(SSU_ERR_INVALID, "max_seqlen must be >= 1 (got %d)", T);
  if (T > ssu::kLogitsMaxTokens) return api_fail(SSU_ERR_UNSUPPORTED, "max_seqlen %d exceeds %d", T, ssu::kLogitsMaxTokens);
  const int rc = check_vocab(vocab);
  if (rc != SSU_OK) return rc;
  const int64_t rows = (int64_t)batch * T;
  if (rows > 65535) return api_fail(SSU_ERR_UNSUPPORTED, "batch %d x max_seqlen %d exceeds 65535 rows per call", batch, T);
  if (rows * ssu::logits_pieces(vocab) > (1 << 23))  // a grid's threads fit 32 bits
    return api_fail(SSU_ERR_UNSUPPORTED, "batch %d x max_seqlen %d x vocab %d exceeds 2^23 workgroups of %d values per call", batch, T,
                    vocab, ssu::kLogitsPiece);
  return SSU_OK;
}

size_t bytes_for(int64_t batch, int64_t T, int64_t vocab) { return (size_t)(batch * T * ssu::logits_pieces(vocab)) * sizeof(float2); }

int launched(hipError_t err) {
  return err == hipSuccess ? api_ok() : api_fail(SSU_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(err));
}

}  // namespace

extern "C" {

int ssu_history_count(const ssu_history *history, const ssu_count_args *a, hipStream_t stream) {
  if (!history) return api_fail(SSU_ERR_INVALID, "history descriptor is NULL");
  if (!a) return api_fail(SSU_ERR_INVALID, "count descriptor is NULL");
  const int rc = check_history(history);
  if (rc != SSU_OK) return rc;
  if (a->batch < 0) return api_fail(SSU_ERR_INVALID, "batch must be >= 0 (got %d)", a->batch);
  if (a->batch > (1 << 20)) return api_fail(SSU_ERR_UNSUPPORTED, "batch %d exceeds 2^20 entries per call", a->batch);
  if (a->rows < 0) return api_fail(SSU_ERR_INVALID, "rows must be >= 0 (got %d)", a->rows);
  if (a->rows > kMaxCountRows) return api_fail(SSU_ERR_UNSUPPORTED, "rows %d exceeds 2^30", a->rows);
  if (!a->cu_seqlens && a->max_seqlen < 1) return api_fail(SSU_ERR_INVALID, "max_seqlen must be >= 1 (got %d)", a->max_seqlen);
  if (a->batch == 0) return api_ok();
  if (!a->slot_idx || (a->rows > 0 && !a->tokens)) return api_fail(SSU_ERR_INVALID, "slot_idx and tokens must not be NULL");
  if (a->cu_seqlens && a->num_tokens) return api_fail(SSU_ERR_INVALID, "cu_seqlens and num_tokens exclude each other");
  if (!a->cu_seqlens && (int64_t)a->batch * a->max_seqlen > a->rows)
    return api_fail(SSU_ERR_INVALID, "rows %d hold no %d entries of %d tokens", a->rows, a->batch, a->max_seqlen);
  if (!aligned(a->slot_idx, 4) || !aligned(a->tokens, 4) || !aligned(a->num_tokens, 4) || !aligned(a->cu_seqlens, 4))
    return api_fail(SSU_ERR_INVALID, "slot_idx, tokens, num_tokens and cu_seqlens must be 4-byte aligned");
  ssu::KCount c;
  c.batch = a->batch;
  c.T = a->cu_seqlens ? 0 : a->max_seqlen;
  c.rows = a->rows;
  c.slot_idx = a->slot_idx;
  c.tokens = a->tokens;
  c.num = a->num_tokens;
  c.cu = a->cu_seqlens;
  c.prompt = a->prompt ? 1 : 0;
  c.reset = a->reset ? 1 : 0;
  return launched(ssu::launch_count(khistory(history), c, stream));
}

size_t ssu_logits_workspace_size(int32_t batch, int32_t max_seqlen, int32_t vocab) {
  if (check_sizes(batch, max_seqlen, vocab) != SSU_OK) return 0;
  api_ok();
  return bytes_for(batch, max_seqlen, vocab);
}

int ssu_logits(const ssu_history *history, const ssu_logits_args *a, hipStream_t stream) {
  if (!a) return api_fail(SSU_ERR_INVALID, "logits descriptor is NULL");
  int rc = check_sizes(a->batch, a->max_seqlen, a->vocab);
  if (rc == SSU_OK && history) rc = check_history(history);
  if (rc != SSU_OK) return rc;
  if (history && history->vocab != a->vocab)
    return api_fail(SSU_ERR_INVALID, "the history is of %d tokens, the logits of %d", history->vocab, a->vocab);
  if (!history && (a->repetition || a->frequency || a->presence))
    return api_fail(SSU_ERR_INVALID, "repetition, frequency and presence need a history");
  const int it = logit_type(raw(a->logits_dtype)), ot = logit_type(raw(a->out_dtype));
  if (it < 0 || ot < 0) return api_fail(SSU_ERR_UNSUPPORTED, "logits_dtype and out_dtype must be SSU_F32, SSU_BF16 or SSU_F16");
  if (a->rows < 0) return api_fail(SSU_ERR_INVALID, "rows must be >= 0 (got %d)", a->rows);
  if (a->batch == 0) return api_ok();
  if (!a->cu_seqlens && (int64_t)a->batch * a->max_seqlen > a->rows)
    return api_fail(SSU_ERR_INVALID, "rows %d hold no %d entries of %d tokens", a->rows, a->batch, a->max_seqlen);
  if (a->rows > 0 && (!a->logits || !a->out)) return api_fail(SSU_ERR_INVALID, "logits and out must not be NULL");
  if (history && !a->slot_idx) return api_fail(SSU_ERR_INVALID, "slot_idx must not be NULL with a history");
  const int isz = it == ssu::kLF32 ? 4 : 2, osz = ot == ssu::kLF32 ? 4 : 2;
  if (!aligned(a->logits, isz) || !aligned(a->out, osz)) return api_fail(SSU_ERR_INVALID, "logits and out must be aligned to their type");
  if (a->logits_row_stride < a->vocab || a->out_row_stride < a->vocab)
    return api_fail(SSU_ERR_INVALID, "row strides %lld and %lld must be at least vocab (%d)", (long long)a->logits_row_stride,
                    (long long)a->out_row_stride, a->vocab);
  if (a->logits == a->out && (it != ot || a->logits_row_stride != a->out_row_stride))
    return api_fail(SSU_ERR_INVALID, "logits written in place must keep their type and row stride");
  if (!aligned(a->cu_seqlens, 4) || !aligned(a->slot_idx, 4) || !aligned(a->tokens, 4) || !aligned(a->temperature, 4) ||
      !aligned(a->repetition, 4) || !aligned(a->frequency, 4) || !aligned(a->presence, 4) || !aligned(a->bias_offsets, 4) ||
      !aligned(a->bias_tokens, 4) || !aligned(a->bias_values, 4) || !aligned(a->mask, 4) || !aligned(a->status, 4))
    return api_fail(SSU_ERR_INVALID, "index arrays, parameters, biases, mask and status must be 4-byte aligned");
  if (a->bias_count < 0 || a->bias_count >= (1 << 24))
    return api_fail(SSU_ERR_INVALID, "bias_count must be in [0, 2^24) (got %d)", a->bias_count);
  if (a->bias_offsets && a->bias_count > 0 && (!a->bias_tokens || !a->bias_values))
    return api_fail(SSU_ERR_INVALID, "bias_tokens and bias_values must not be NULL with bias_offsets");
  if (a->mask && a->mask_row_stride != 0 && a->mask_row_stride < (a->vocab + 31) / 32)
    return api_fail(SSU_ERR_INVALID, "mask_row_stride %lld must be 0 or at least %d words", (long long)a->mask_row_stride,
                    (a->vocab + 31) / 32);
  if (!a->no_softmax) {
    const size_t need = bytes_for(a->batch, a->max_seqlen, a->vocab);
    if (!a->workspace || a->workspace_bytes < need)
      return api_fail(SSU_ERR_WORKSPACE, "the logits need a workspace of %zu bytes (got %zu%s)", need, a->workspace_bytes,
                      a->workspace ? "" : ", NULL");
    if (!aligned(a->workspace, 16)) return api_fail(SSU_ERR_INVALID, "workspace must be 16-byte aligned");
  }
  ssu::KLogits l;
  l.batch = a->batch;
  l.T = a->max_seqlen;
  l.rows = a->rows;
  l.vocab = a->vocab;
  l.in = static_cast<const uint8_t *>(a->logits);
  l.in_stride = a->logits_row_stride * isz;
  l.out = static_cast<uint8_t *>(a->out);
  l.out_stride = a->out_row_stride * osz;
  l.cu = a->cu_seqlens;
  l.slot_idx = a->slot_idx;
  l.tokens = a->tokens;
  l.temperature = a->temperature;
  l.repetition = a->repetition;
  l.frequency = a->frequency;
  l.presence = a->presence;
  l.bias_off = a->bias_count > 0 ? a->bias_offsets : nullptr;
  l.bias_tok = a->bias_tokens;
  l.bias_val = a->bias_values;
  l.bias_count = a->bias_count;
  l.mask = a->mask;
  l.mask_stride = a->mask_row_stride;
  l.ws = static_cast<float2 *>(a->workspace);
  l.status = a->status;
  // What is more than the last cache's 256 MiB would only push itself out of it (bf16 rows of 131072 values, 512 of them
  // 88 -> 76 us, 1024 185 -> 159; f32 ones 187 -> 153; 256 bf16 rows 45.7 -> 46.1), and less is there for who reads it next.
  l.past = (int64_t)a->rows * a->vocab * (isz + osz) >= (int64_t)256 << 20;
  return launched(ssu::launch_logits(khistory(history), l, it, ot, !a->no_softmax, stream));
}

}  // extern "C"
