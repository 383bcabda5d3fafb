// Host entry points of the gated delta rule (include/ssu_delta.h): argument
// checks and launches.  Nothing here allocates or synchronises.
#include <cstring>

#include <hip/hip_runtime.h>

#include "../../include/ssu_delta.h"
#include "delta_internal.h"

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

constexpr int64_t kWide = (int64_t)1 << 23;

int check_dims(int32_t hk, int32_t hv, int32_t dk, int32_t dv) {
  if (hk < 1 || hv < 1) return api_fail(SSU_ERR_INVALID, "nheads_k and nheads_v must be positive (got %d, %d)", hk, hv);
  if (hv % hk != 0)
    return api_fail(SSU_ERR_INVALID, "nheads_v (%d) must be a multiple of nheads_k (%d)", hv, hk);
  if (dk != 64 && dk != 128) return api_fail(SSU_ERR_UNSUPPORTED, "dim_k must be 64 or 128 (got %d)", dk);
  if (dv < 16 || dv > ssu::kDeltaMaxDv || dv % 16 != 0)
    return api_fail(SSU_ERR_UNSUPPORTED, "dim_v must be a multiple of 16 in [16, %d] (got %d)", ssu::kDeltaMaxDv, dv);
  if ((int64_t)hv * dv >= kWide)  // a few rows are addressed with 32-bit byte offsets
    return api_fail(SSU_ERR_UNSUPPORTED, "nheads_v x dim_v must be below 2^23 (got %d x %d)", hv, dv);
  return SSU_OK;
}

int64_t state_bytes(int32_t t) { return t == SSU_F32 ? 4 : 2; }

int check_cache(const ssu_delta_cache *c) {
  if (!c) return api_fail(SSU_ERR_INVALID, "cache descriptor is NULL");
  if (c->num_slots < 1) return api_fail(SSU_ERR_INVALID, "num_slots must be positive (got %d)", c->num_slots);
  const int rc = check_dims(c->nheads_k, c->nheads_v, c->dim_k, c->dim_v);
  if (rc != SSU_OK) return rc;
  if (c->ring_len < 1 || c->ring_len > ssu::kMaxRing)
    return api_fail(SSU_ERR_UNSUPPORTED, "ring_len must be in [1, %d] (got %d)", ssu::kMaxRing, c->ring_len);
  const int32_t sd = raw(c->state_dtype);
  if (sd != SSU_F32 && sd != SSU_BF16 && sd != SSU_F16)
    return api_fail(sd == SSU_FP8_E4M3 || sd == SSU_NVFP4 ? SSU_ERR_UNSUPPORTED : SSU_ERR_INVALID,
                    "state_dtype must be SSU_F32, SSU_BF16 or SSU_F16 (got %d)", sd);
  if (raw(c->io_dtype) != SSU_BF16) return api_fail(SSU_ERR_UNSUPPORTED, "io_dtype must be SSU_BF16 (q, k, v and their rings)");
  if (!c->state || !c->k_cache || !c->v_cache || !c->gate_cache || !c->ring_start)
    return api_fail(SSU_ERR_INVALID, "cache tensors must not be NULL");
  if (!aligned(c->state, 16) || !aligned(c->k_cache, 16) || !aligned(c->v_cache, 16) || !aligned(c->gate_cache, 8) ||
      !aligned(c->ring_start, 4) || !aligned(c->status, 4))
    return api_fail(SSU_ERR_INVALID, "cache pointers must be 16-byte aligned (gate_cache: 8-byte; ring_start, status: 4-byte)");
  const int64_t hk = c->nheads_k, hv = c->nheads_v, L = c->ring_len;
  const struct {
    const char *name;
    int64_t stride, need, unit;
  } s[] = {
      {"state", c->state_slot_stride, hv * c->dim_v * c->dim_k * state_bytes(sd), 16},
      {"k_cache", c->k_slot_stride, hk * L * c->dim_k * 2, 16},
      {"v_cache", c->v_slot_stride, hv * L * c->dim_v * 2, 16},
      {"gate_cache", c->gate_slot_stride, hv * L * 8, 8},
  };
  for (const auto &t : s) {
    if (t.stride < t.need)
      return api_fail(SSU_ERR_INVALID, "%s slot stride %lld is smaller than one packed slot (%lld bytes)", t.name,
                      (long long)t.stride, (long long)t.need);
    if (t.stride % t.unit != 0)
      return api_fail(SSU_ERR_INVALID, "%s slot stride %lld is not a multiple of %lld bytes", t.name, (long long)t.stride,
                      (long long)t.unit);
  }
  return SSU_OK;
}

int check_pairs(int64_t n, int64_t heads, const char *what) {
  if (n < 0) return api_fail(SSU_ERR_INVALID, "%s must be >= 0 (got %lld)", what, (long long)n);
  if (n * heads > SSU_DELTA_MAX_PAIRS)
    return api_fail(SSU_ERR_UNSUPPORTED, "%s %lld x %lld heads exceeds SSU_DELTA_MAX_PAIRS (%d) (entry, head) pairs per call",
                    what, (long long)n, (long long)heads, SSU_DELTA_MAX_PAIRS);
  return SSU_OK;
}

int check_row_stride(const char *name, int64_t stride, int64_t packed) {
  if (stride < packed || stride % 8 != 0)
    return api_fail(SSU_ERR_INVALID, "%s_row_stride %lld must be a multiple of 8 elements and at least %lld", name,
                    (long long)stride, (long long)packed);
  return SSU_OK;
}

// q, k, v and the gate inputs, which a step and a prompt have alike.
template <class A>
int check_inputs(const A *a, bool rows, int64_t hk, int64_t hv, int64_t dk, int64_t dv) {
  if (!a->A || !a->dt_bias) return api_fail(SSU_ERR_INVALID, "A and dt_bias must not be NULL");
  if (rows && (!a->q || !a->k || !a->v || !a->dt || !a->beta || !a->out))
    return api_fail(SSU_ERR_INVALID, "q, k, v, dt, beta and out must not be NULL");
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 16))
    return api_fail(SSU_ERR_INVALID, "q, k, v and out must be 16-byte aligned");
  if (!aligned(a->dt, 4) || !aligned(a->beta, 4) || !aligned(a->A, 4) || !aligned(a->dt_bias, 4))
    return api_fail(SSU_ERR_INVALID, "dt, beta, A and dt_bias must be 4-byte aligned");
  int rc = check_row_stride("q", a->q_row_stride, hk * dk);
  if (rc == SSU_OK) rc = check_row_stride("k", a->k_row_stride, hk * dk);
  if (rc == SSU_OK) rc = check_row_stride("v", a->v_row_stride, hv * dv);
  if (rc != SSU_OK) return rc;
  const int32_t od = raw(a->out_dtype);
  if (od != SSU_BF16 && od != SSU_F32) return api_fail(SSU_ERR_UNSUPPORTED, "out_dtype must be SSU_BF16 or SSU_F32");
  return SSU_OK;
}

ssu::DCache dcache(const ssu_delta_cache *c) {
  ssu::DCache k;
  k.state = static_cast<uint8_t *>(c->state);
  k.state_stride = c->state_slot_stride;
  k.kc = static_cast<uint8_t *>(c->k_cache);
  k.k_stride = c->k_slot_stride;
  k.vc = static_cast<uint8_t *>(c->v_cache);
  k.v_stride = c->v_slot_stride;
  k.gc = reinterpret_cast<uint8_t *>(c->gate_cache);
  k.g_stride = c->gate_slot_stride;
  k.ring_start = c->ring_start;
  k.status = c->status;
  k.num_slots = c->num_slots;
  k.Hk = c->nheads_k;
  k.Hv = c->nheads_v;
  k.hpg = c->nheads_v / c->nheads_k;
  k.dk = c->dim_k;
  k.dv = c->dim_v;
  k.L = c->ring_len;
  k.norm = c->no_qk_norm ? 0 : 1;
  return k;
}

int launched(hipError_t err) {
  return err == hipSuccess ? api_ok() : api_fail(SSU_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(err));
}

#define SSU_DELTA_ST(FN, ...)                                                   \
  (raw(cache->state_dtype) == SSU_F32    ? ssu::FN<ssu::kF32>(__VA_ARGS__)      \
   : raw(cache->state_dtype) == SSU_BF16 ? ssu::FN<ssu::kBF16>(__VA_ARGS__)     \
                                         : ssu::FN<ssu::kF16>(__VA_ARGS__))

// The states argument of init and read.
int check_states(const ssu_delta_cache *c, const float *states, int64_t stride, const int32_t *slot_idx, bool read) {
  const int64_t packed = (int64_t)c->nheads_v * c->dim_v * c->dim_k;
  if (!states || !slot_idx) return api_fail(SSU_ERR_INVALID, "states and slot_idx must not be NULL");
  if (stride < 0 || stride % 4 != 0 || (stride < packed && (read || stride != 0)))
    return api_fail(SSU_ERR_INVALID, "states_batch_stride %lld must be a multiple of 4 and at least one packed state (%lld)%s",
                    (long long)stride, (long long)packed, read ? "" : ", or 0");
  if (!aligned(states, 16) || !aligned(slot_idx, 4))
    return api_fail(SSU_ERR_INVALID, "states must be 16-byte aligned, slot_idx 4-byte");
  return SSU_OK;
}

constexpr int64_t kMaxItems = (int64_t)1 << 30;  // rows x heads

int check_prefill_sizes(int64_t rows, int64_t n, int64_t hv) {
  if (rows < 0) return api_fail(SSU_ERR_INVALID, "rows must be >= 0 (got %lld)", (long long)rows);
  if (hv < 1) return api_fail(SSU_ERR_INVALID, "nheads_v must be positive (got %lld)", (long long)hv);
  const int rc = check_pairs(n, hv, "num_seqs");
  if (rc != SSU_OK) return rc;
  if (rows * hv > kMaxItems)
    return api_fail(SSU_ERR_UNSUPPORTED, "rows %lld x nheads_v %lld exceeds 2^30", (long long)rows, (long long)hv);
  return SSU_OK;
}

size_t prefill_bytes(int64_t rows, int64_t n, int64_t hv) {
  return (size_t)((rows / ssu::kChunk + n) * hv * ssu::kRecMax);
}

}  // namespace

extern "C" {

int ssu_delta_replay_step(const ssu_delta_cache *cache, const ssu_delta_step *s, hipStream_t stream) {
  int rc = check_cache(cache);
  if (rc != SSU_OK) return rc;
  if (!s) return api_fail(SSU_ERR_INVALID, "step descriptor is NULL");
  const int tmax = cache->ring_len < ssu::kMaxTokens ? cache->ring_len : ssu::kMaxTokens;
  if (s->max_seqlen < 1 || s->max_seqlen > tmax)
    return api_fail(s->max_seqlen < 1 || s->max_seqlen > cache->ring_len ? SSU_ERR_INVALID : SSU_ERR_UNSUPPORTED,
                    "max_seqlen %d must be in [1, min(16, ring_len) = %d]", s->max_seqlen, tmax);
  rc = check_pairs(s->batch, cache->nheads_v, "batch");
  if (rc != SSU_OK) return rc;
  if (s->batch == 0) return api_ok();
  if (!s->slot_idx || !s->prev_num_accepted)
    return api_fail(SSU_ERR_INVALID, "slot_idx and prev_num_accepted must not be NULL");
  if (!aligned(s->slot_idx, 4) || !aligned(s->prev_num_accepted, 4) || !aligned(s->cu_seqlens, 4))
    return api_fail(SSU_ERR_INVALID, "the index arrays must be 4-byte aligned");
  rc = check_inputs(s, true, cache->nheads_k, cache->nheads_v, cache->dim_k, cache->dim_v);
  if (rc != SSU_OK) return rc;
  ssu::DStep k;
  k.batch = s->batch;
  k.T = s->max_seqlen;
  k.slot_idx = s->slot_idx;
  k.pnat = s->prev_num_accepted;
  k.cu = s->cu_seqlens;
  k.q = static_cast<const uint16_t *>(s->q);
  k.k = static_cast<const uint16_t *>(s->k);
  k.v = static_cast<const uint16_t *>(s->v);
  k.q_stride = s->q_row_stride;
  k.k_stride = s->k_row_stride;
  k.v_stride = s->v_row_stride;
  k.dt = s->dt;
  k.beta = s->beta;
  k.A = s->A;
  k.dt_bias = s->dt_bias;
  k.scale = s->scale;
  k.softplus = s->no_dt_softplus ? 0 : 1;
  k.sigmoid = s->no_beta_sigmoid ? 0 : 1;
  k.out = s->out;
  const int ot = raw(s->out_dtype) == SSU_F32 ? ssu::kOutF32 : ssu::kOutBF16;
  return launched(SSU_DELTA_ST(delta_step_st, dcache(cache), k, ot, stream));
}

int ssu_delta_flush(const ssu_delta_cache *cache, const int32_t *slot_idx, const int32_t *num_fold, int32_t n,
                    hipStream_t stream) {
  int rc = check_cache(cache);
  if (rc == SSU_OK) rc = check_pairs(n, cache->nheads_v, "n");
  if (rc != SSU_OK) return rc;
  if (n == 0) return api_ok();
  if (!slot_idx || !num_fold) return api_fail(SSU_ERR_INVALID, "slot_idx and num_fold must not be NULL");
  if (!aligned(slot_idx, 4) || !aligned(num_fold, 4))
    return api_fail(SSU_ERR_INVALID, "slot_idx and num_fold must be 4-byte aligned");
  return launched(SSU_DELTA_ST(delta_flush_st, dcache(cache), slot_idx, num_fold, n, stream));
}

int ssu_delta_init_state(const ssu_delta_cache *cache, const float *states, int64_t states_batch_stride,
                         const int32_t *slot_idx, int32_t n, hipStream_t stream) {
  int rc = check_cache(cache);
  if (rc == SSU_OK) rc = check_pairs(n, cache->nheads_v, "n");
  if (rc != SSU_OK) return rc;
  if (n == 0) return api_ok();
  rc = check_states(cache, states, states_batch_stride, slot_idx, false);
  if (rc != SSU_OK) return rc;
  return launched(SSU_DELTA_ST(delta_init_st, dcache(cache), states, states_batch_stride, slot_idx, n, stream));
}

int ssu_delta_read_state(const ssu_delta_cache *cache, float *states, int64_t states_batch_stride,
                         const int32_t *slot_idx, int32_t n, hipStream_t stream) {
  int rc = check_cache(cache);
  if (rc == SSU_OK) rc = check_pairs(n, cache->nheads_v, "n");
  if (rc != SSU_OK) return rc;
  if (n == 0) return api_ok();
  rc = check_states(cache, states, states_batch_stride, slot_idx, true);
  if (rc != SSU_OK) return rc;
  return launched(SSU_DELTA_ST(delta_read_st, dcache(cache), states, states_batch_stride, slot_idx, n, stream));
}

size_t ssu_delta_prefill_workspace_size(int32_t rows, int32_t num_seqs, int32_t nheads_v) {
  if (check_prefill_sizes(rows, num_seqs, nheads_v) != SSU_OK) return 0;
  api_ok();
  return prefill_bytes(rows, num_seqs, nheads_v);
}

int ssu_delta_prefill(const ssu_delta_prefill_args *a, hipStream_t stream) {
  if (!a) return api_fail(SSU_ERR_INVALID, "prefill descriptor is NULL");
  int rc = check_dims(a->nheads_k, a->nheads_v, a->dim_k, a->dim_v);
  if (rc == SSU_OK) rc = check_prefill_sizes(a->rows, a->num_seqs, a->nheads_v);
  if (rc != SSU_OK) return rc;
  if (raw(a->io_dtype) != SSU_BF16) return api_fail(SSU_ERR_UNSUPPORTED, "io_dtype must be SSU_BF16 (q, k and v)");
  if (a->num_seqs == 0) return api_ok();
  if (!a->cu_seqlens) return api_fail(SSU_ERR_INVALID, "cu_seqlens must not be NULL");
  if (!aligned(a->cu_seqlens, 4) || !aligned(a->status, 4))
    return api_fail(SSU_ERR_INVALID, "cu_seqlens and status must be 4-byte aligned");
  if (!aligned(a->initial_states, 16) || !aligned(a->final_states, 16))
    return api_fail(SSU_ERR_INVALID, "initial_states and final_states must be 16-byte aligned");
  rc = check_inputs(a, a->rows > 0, a->nheads_k, a->nheads_v, a->dim_k, a->dim_v);
  if (rc != SSU_OK) return rc;
  if (a->q_row_stride >= kWide || a->k_row_stride >= kWide || a->v_row_stride >= kWide)  // as in check_dims
    return api_fail(SSU_ERR_UNSUPPORTED, "the row strides must be below 2^23 elements");
  const size_t need = prefill_bytes(a->rows, a->num_seqs, a->nheads_v);
  if (!a->workspace || a->workspace_bytes < need)
    return api_fail(SSU_ERR_WORKSPACE, "the prefill needs a workspace of %zu bytes (got %zu%s)", need, a->workspace_bytes,
                    a->workspace ? "" : ", NULL");
  if (!aligned(a->workspace, 16)) return api_fail(SSU_ERR_INVALID, "workspace must be 16-byte aligned");
  ssu::DPrefill p;
  p.n = a->num_seqs;
  p.rows = a->rows;
  p.Hk = a->nheads_k;
  p.Hv = a->nheads_v;
  p.hpg = a->nheads_v / a->nheads_k;
  p.dk = a->dim_k;
  p.dv = a->dim_v;
  p.cu = a->cu_seqlens;
  p.q = static_cast<const uint16_t *>(a->q);
  p.k = static_cast<const uint16_t *>(a->k);
  p.v = static_cast<const uint16_t *>(a->v);
  p.q_stride = a->q_row_stride;
  p.k_stride = a->k_row_stride;
  p.v_stride = a->v_row_stride;
  p.dt = a->dt;
  p.beta = a->beta;
  p.A = a->A;
  p.dt_bias = a->dt_bias;
  p.scale = a->scale;
  p.softplus = a->no_dt_softplus ? 0 : 1;
  p.sigmoid = a->no_beta_sigmoid ? 0 : 1;
  p.norm = a->no_qk_norm ? 0 : 1;
  p.h0 = a->initial_states;
  p.h1 = a->final_states;
  p.out = a->out;
  p.ws = static_cast<uint8_t *>(a->workspace);
  p.status = a->status;
  return launched(ssu::launch_delta_prefill(p, raw(a->out_dtype) == SSU_F32 ? ssu::kOutF32 : ssu::kOutBF16, stream));
}

}  // extern "C"
