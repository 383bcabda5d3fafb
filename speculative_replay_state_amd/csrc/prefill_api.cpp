// Host entry points of prompts under the selective state update
// (include/ssu_prefill.h): argument checks and the launch.
#include <cstring>

#include <hip/hip_runtime.h>

#include "../../include/ssu_prefill.h"
#include "prefill_internal.h"

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

constexpr int64_t kWide = (int64_t)1 << 23;      // elements between rows: a chunk's rows are addressed with 32-bit byte offsets
constexpr int64_t kMaxItems = (int64_t)1 << 30;  // rows x heads
constexpr int64_t kMaxPairs = (int64_t)1 << 20;  // sequences x heads: every launch grid, in threads, then fits 32 bits
constexpr int32_t kMaxHeads = 32768;

int check_sizes(int64_t rows, int64_t n, int64_t heads) {
  if (rows < 0) return api_fail(SSU_ERR_INVALID, "rows must be >= 0 (got %lld)", (long long)rows);
  if (n < 0) return api_fail(SSU_ERR_INVALID, "num_seqs must be >= 0 (got %lld)", (long long)n);
  if (heads < 1) return api_fail(SSU_ERR_INVALID, "nheads must be positive (got %lld)", (long long)heads);
  if (heads > kMaxHeads) return api_fail(SSU_ERR_UNSUPPORTED, "nheads %lld exceeds %d", (long long)heads, kMaxHeads);
  if (n * heads > kMaxPairs)
    return api_fail(SSU_ERR_UNSUPPORTED, "num_seqs %lld x nheads %lld exceeds 2^20 (sequence, head) pairs per call", (long long)n,
                    (long long)heads);
  if (rows * heads > kMaxItems)
    return api_fail(SSU_ERR_UNSUPPORTED, "rows %lld x nheads %lld exceeds 2^30", (long long)rows, (long long)heads);
  return SSU_OK;
}

// States of the segments, then their decays.
size_t state_bytes(int64_t slots, int64_t heads) { return (size_t)(slots * heads * ssu::kHeadDim * ssu::kDState) * sizeof(float); }
size_t bytes_for(int64_t slots, int64_t heads) { return state_bytes(slots, heads) + (size_t)(slots * heads) * sizeof(double); }

int check_row_stride(const char *name, int64_t stride, int64_t packed) {
  if (stride < packed || stride % 8 != 0)
    return api_fail(SSU_ERR_INVALID, "%s_row_stride %lld must be a multiple of 8 elements and at least %lld", name,
                    (long long)stride, (long long)packed);
  if (stride >= kWide) return api_fail(SSU_ERR_UNSUPPORTED, "the row strides must be below 2^23 elements (%s: %lld)", name, (long long)stride);
  return SSU_OK;
}

}  // namespace

extern "C" {

size_t ssu_prefill_workspace_size(int32_t rows, int32_t num_seqs, int32_t nheads) {
  if (check_sizes(rows, num_seqs, nheads) != SSU_OK) return 0;
  api_ok();
  // (of any call of up to as many rows and sequences; none where no sequence can have two segments)
  return rows <= 2 * ssu::kLeastSegment ? 0 : bytes_for(ssu::prefill_most_slots(rows, num_seqs, nheads), nheads);
}

int ssu_prefill(const ssu_prefill_args *a, hipStream_t stream) {
  if (!a) return api_fail(SSU_ERR_INVALID, "prefill descriptor is NULL");
  if (a->ngroups < 1) return api_fail(SSU_ERR_INVALID, "ngroups must be positive (got %d)", a->ngroups);
  int rc = check_sizes(a->rows, a->num_seqs, a->nheads);
  if (rc != SSU_OK) return rc;
  if (a->nheads % a->ngroups != 0)
    return api_fail(SSU_ERR_INVALID, "nheads (%d) must be a multiple of ngroups (%d)", a->nheads, a->ngroups);
  if (a->headdim != ssu::kHeadDim || a->dstate != ssu::kDState)
    return api_fail(SSU_ERR_UNSUPPORTED, "only headdim 64 and dstate 128 are implemented (got %d, %d)", a->headdim, a->dstate);
  if (raw(a->io_dtype) != SSU_BF16) return api_fail(SSU_ERR_UNSUPPORTED, "io_dtype must be SSU_BF16 (x, B, C and z)");
  const int32_t od = raw(a->out_dtype);
  if (od != SSU_BF16 && od != SSU_F32) return api_fail(SSU_ERR_UNSUPPORTED, "out_dtype must be SSU_BF16 or SSU_F32");
  if (a->num_seqs == 0) return api_ok();
  if (!a->cu_seqlens || !a->A || !a->D || !a->dt_bias)
    return api_fail(SSU_ERR_INVALID, "cu_seqlens, A, D and dt_bias must not be NULL");
  if (a->rows > 0 && (!a->x || !a->B || !a->C || !a->dt || !a->out))
    return api_fail(SSU_ERR_INVALID, "x, B, C, dt and out must not be NULL");
  if (!aligned(a->x, 16) || !aligned(a->B, 16) || !aligned(a->C, 16) || !aligned(a->z, 16) || !aligned(a->out, 16) ||
      !aligned(a->initial_states, 16) || !aligned(a->final_states, 16))
    return api_fail(SSU_ERR_INVALID, "x, B, C, z, out and the states must be 16-byte aligned");
  if (!aligned(a->dt, 4) || !aligned(a->A, 4) || !aligned(a->D, 4) || !aligned(a->dt_bias, 4) || !aligned(a->cu_seqlens, 4) ||
      !aligned(a->status, 4))
    return api_fail(SSU_ERR_INVALID, "dt, A, D, dt_bias, cu_seqlens and status must be 4-byte aligned");
  const int64_t inner = (int64_t)a->nheads * ssu::kHeadDim, group = (int64_t)a->ngroups * ssu::kDState;
  rc = check_row_stride("x", a->x_row_stride, inner);
  if (rc == SSU_OK) rc = check_row_stride("B", a->B_row_stride, group);
  if (rc == SSU_OK) rc = check_row_stride("C", a->C_row_stride, group);
  if (rc == SSU_OK && a->z) rc = check_row_stride("z", a->z_row_stride, inner);
  if (rc != SSU_OK) return rc;
  const int seg = ssu::prefill_segment(a->rows, a->num_seqs, a->nheads);
  const int64_t slots = a->rows <= 2 * (int64_t)seg ? 0 : ssu::prefill_slots(a->rows, a->num_seqs, seg);
  const size_t need = bytes_for(slots, a->nheads);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need))
    return api_fail(SSU_ERR_WORKSPACE, "the prefill needs a workspace of %zu bytes (got %zu%s)", need, a->workspace_bytes,
                    a->workspace ? "" : ", NULL");
  if (!aligned(a->workspace, 16)) return api_fail(SSU_ERR_INVALID, "workspace must be 16-byte aligned");
  ssu::KPrefill p;
  p.n = a->num_seqs;
  p.rows = a->rows;
  p.H = a->nheads;
  p.G = a->ngroups;
  p.hpg = a->nheads / a->ngroups;
  p.seg = seg;
  p.cu = a->cu_seqlens;
  p.x = static_cast<const uint16_t *>(a->x);
  p.B = static_cast<const uint16_t *>(a->B);
  p.C = static_cast<const uint16_t *>(a->C);
  p.z = static_cast<const uint16_t *>(a->z);
  p.x_stride = a->x_row_stride;
  p.B_stride = a->B_row_stride;
  p.C_stride = a->C_row_stride;
  p.z_stride = a->z_row_stride;
  p.dt = a->dt;
  p.A = a->A;
  p.D = a->D;
  p.dt_bias = a->dt_bias;
  p.softplus = a->no_dt_softplus ? 0 : 1;
  p.h0 = a->initial_states;
  p.h1 = a->final_states;
  p.out = a->out;
  p.ws = static_cast<float *>(a->workspace);
  p.decay = reinterpret_cast<double *>(static_cast<uint8_t *>(a->workspace) + state_bytes(slots, a->nheads));
  p.status = a->status;
  const hipError_t err = ssu::launch_prefill(p, od == SSU_F32 ? ssu::kOutF32 : ssu::kOutBF16, stream);
  return err == hipSuccess ? api_ok() : api_fail(SSU_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(err));
}

}  // extern "C"
