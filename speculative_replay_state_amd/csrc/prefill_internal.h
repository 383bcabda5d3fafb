// Internal interface between the host entry points of prompts under the
// selective state update (prefill_api.cpp, ssu_api.cpp) and their kernels
// (prefill.hip, read_kernels.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "ssu_internal.h"

namespace ssu {

constexpr int kPChunk = 64;  // tokens of a chunk

struct KPrefill {
  int n, rows, H, G, hpg;
  int seg;  // tokens of a segment, a multiple of kPChunk
  const int32_t *cu;
  const uint16_t *x, *B, *C, *z;
  int64_t x_stride, B_stride, C_stride, z_stride;  // elements between rows
  const float *dt, *A, *D, *dt_bias;
  int softplus;
  const float *h0;
  float *h1;
  void *out;
  float *ws;      // [slot][H][64 * 128]: a segment's own update of the state, later the state it starts from
  double *decay;  // [slot][H]: log2 of a segment's whole decay
  int32_t *status;
};

// Segment slots: sequence s has slots cu[s] / seg + s and on, as many as segments.
constexpr int64_t prefill_slots(int64_t rows, int64_t n, int64_t seg) { return rows / seg + n; }
constexpr int kLeastSegment = 256;
int prefill_segment(int64_t rows, int64_t n, int64_t heads);
int64_t prefill_most_slots(int64_t rows, int64_t n, int64_t heads);

hipError_t launch_prefill(const KPrefill &p, int out_type, hipStream_t stream);
hipError_t launch_read(const KCache &c, float *states, int64_t stride, const int32_t *slot_idx, int n, int state_type, int recur,
                       hipStream_t stream);

}  // namespace ssu
