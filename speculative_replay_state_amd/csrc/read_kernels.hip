// Checkpoints as fp32 states (ssu_read_state).
//
// A wave takes a row block of 16 rows; a lane 4 neighbouring values of a row,
// so that a store instruction writes 1 KiB in one piece: the stores are as many bytes as
// the loads (fp32) to 8 times as many, and the loads find the row block's other lines in
// the CU's cache.  HBM bounds it: 64 slots of 128 heads of fp8, 338 MB, take 66 us, a
// copy's 5.1 TB/s; one slot of 16 heads takes 3.0.
#include "prefill_internal.h"
#include "ssu_device.cuh"

namespace ssu {

namespace {

constexpr int kRowBlocks = kHeadDim / 16;
constexpr int kHeadValues = kHeadDim * kDState;
constexpr int read_bits(int ST) { return ST == kF32 ? 32 : (ST == kFP8 ? 8 : (ST == kNVFP4 ? 4 : 16)); }

// Four values from their 4 * bits bits, before any scale.
template <int ST>
__device__ __forceinline__ f32x4 four(const uint8_t *p) {
  if constexpr (ST == kF32) return *reinterpret_cast<const f32x4 *>(p);
  if constexpr (ST == kBF16 || ST == kF16) {
    const u32x2 w = ld8(p);
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
      v[i] = ST == kBF16 ? bf2f(b) : (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    }
    return v;
  }
  if constexpr (ST == kFP8) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    return f32x4{a[0], a[1], b[0], b[1]};
  }
  const uint32_t w = *reinterpret_cast<const uint16_t *>(p);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  return f32x4{a[0], a[1], b[0], b[1]};
}

// `state`: the checkpoint's pages (or the recurrence one's).
template <int ST>
__global__ __launch_bounds__(kRowBlocks * 64) void read_kernel(KCache c, const uint8_t *state, int64_t state_stride, float *states,
                                                               int64_t stride, const int32_t *slot_idx) {
  const int j = blockIdx.x / c.H, h = blockIdx.x - j * c.H, slot = slot_idx[j];
  if (slot <= 0 || slot >= c.num_slots) return;
  const int rb = threadIdx.x >> 6, lane = threadIdx.x & 63;
  constexpr int kUnits = 128 / read_bits(ST);               // values of a 16-byte chunk
  constexpr int kHeadBytes = kHeadValues * read_bits(ST) / 8, kBlock = kHeadBytes / kRowBlocks;
  const uint8_t *block = state + (int64_t)slot * state_stride + (int64_t)h * kHeadBytes + rb * kBlock;
  float *to = states + (int64_t)j * stride + (int64_t)h * kHeadValues + rb * 16 * kDState;
  const float g = ST == kNVFP4 ? *reinterpret_cast<const float *>(c.gw + (int64_t)slot * c.gw_stride) : 1.f;
  f32x4 v[8];
  float scale[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // row m, values n .. n + 3: quarter q, chunk u of lane 16 q + m
    const int m = 2 * i + (lane >> 5), n = 4 * (lane & 31), q = n >> 5, t = n & 31, l = 16 * q + m;
    v[i] = four<ST>(block + (t / kUnits * 64 + l) * 16 + t % kUnits * read_bits(ST) / 8);
    scale[i] = 1.f;
    if constexpr (ST == kFP8)
      scale[i] = reinterpret_cast<const float *>(c.scale + (int64_t)slot * c.scale_stride)[h * kHeadDim + 16 * rb + m];
    if constexpr (ST == kNVFP4)
      scale[i] = __builtin_amdgcn_cvt_f32_fp8(
          c.scale[(int64_t)slot * c.scale_stride + (int64_t)h * (kHeadValues / 16) + l * 8 + rb * 2 + (t >> 4)], 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (ST == kFP8) v[i][e] *= scale[i];
      if constexpr (ST == kNVFP4) v[i][e] = v[i][e] * scale[i] * g;
    }
    *reinterpret_cast<f32x4 *>(to + i * 256 + lane * 4) = v[i];
  }
}

}  // namespace

hipError_t launch_read(const KCache &c, float *states, int64_t stride, const int32_t *slot_idx, int n, int state_type, int recur,
                       hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)n * c.H)), block(kRowBlocks * 64);
  const uint8_t *state = recur ? c.recur : c.state;
  const int64_t page = recur ? c.recur_stride : c.state_stride;
  switch (recur ? kF16 : state_type) {
    case kF32: read_kernel<kF32><<<grid, block, 0, st>>>(c, state, page, states, stride, slot_idx); break;
    case kBF16: read_kernel<kBF16><<<grid, block, 0, st>>>(c, state, page, states, stride, slot_idx); break;
    case kF16: read_kernel<kF16><<<grid, block, 0, st>>>(c, state, page, states, stride, slot_idx); break;
    case kFP8: read_kernel<kFP8><<<grid, block, 0, st>>>(c, state, page, states, stride, slot_idx); break;
    default: read_kernel<kNVFP4><<<grid, block, 0, st>>>(c, state, page, states, stride, slot_idx); break;
  }
  return hipGetLastError();
}

}  // namespace ssu
