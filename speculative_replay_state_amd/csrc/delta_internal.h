// Internal interface between the host entry points of the gated delta rule
// (delta_api.cpp) and its kernels (delta_kernels.cuh, instantiated per state
// type by delta_kernels_inst.hip; the prompt kernels in delta_prefill.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "ssu_internal.h"

namespace ssu {

constexpr float kDeltaEps = 1e-6f;     // under the root of the unit length of q and k
constexpr int kDeltaMaxDv = 256;
constexpr int kChunk = 32;             // tokens of a prompt chunk: one K = 32 MFMA step over tokens

// Scratch of one (chunk, value head): T - I, T = (I + A)^-1, the chunk's factors,
// and P, both triangles as MFMA row operands without their zero upper blocks, in
// two bf16 parts towards bf16 outputs and in three towards fp32 ones.
constexpr int kRecPart = 64 * (8 + 16);  // rows 0..15: 8 bytes a lane; rows 16..31: 16 bytes
constexpr int kRecF = 544;  // f32: b[32], b e^G rk[32], e^(Gw-G) rk[32], scale rq e^G[32], e^Gw
constexpr int rec_t(int parts) { return parts * kRecPart; }
constexpr int rec_bytes(int parts) { return rec_t(parts) + kRecF + parts * kRecPart; }
constexpr int kRecMax = rec_bytes(3);

struct DCache {
  uint8_t *state;
  int64_t state_stride;
  uint8_t *kc;
  int64_t k_stride;
  uint8_t *vc;
  int64_t v_stride;
  uint8_t *gc;
  int64_t g_stride;
  int32_t *ring_start;
  int32_t *status;
  int num_slots, Hk, Hv, hpg, dk, dv, L;
  int norm;  // 1: q and k scaled to unit length
};

struct DStep {
  int batch, T;
  const int32_t *slot_idx;
  const int32_t *pnat;
  const int32_t *cu;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between rows
  const float *dt, *beta, *A, *dt_bias;
  float scale;
  int softplus, sigmoid;
  void *out;
};

struct DPrefill {
  int n, rows, Hk, Hv, hpg, dk, dv;
  const int32_t *cu;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *dt, *beta, *A, *dt_bias;
  float scale;
  int softplus, sigmoid, norm;
  const float *h0;
  float *h1;
  void *out;
  uint8_t *ws;
  int32_t *status;
};

template <int ST>
hipError_t delta_step_st(const DCache &c, const DStep &s, int out_type, hipStream_t stream);
template <int ST>
hipError_t delta_flush_st(const DCache &c, const int32_t *slot_idx, const int32_t *num_fold, int n, hipStream_t stream);
template <int ST>
hipError_t delta_init_st(const DCache &c, const float *states, int64_t stride, const int32_t *slot_idx, int n,
                         hipStream_t stream);
template <int ST>
hipError_t delta_read_st(const DCache &c, float *states, int64_t stride, const int32_t *slot_idx, int n,
                         hipStream_t stream);
hipError_t launch_delta_prefill(const DPrefill &p, int out_type, hipStream_t stream);

}  // namespace ssu
