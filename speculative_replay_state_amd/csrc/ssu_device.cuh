// Small device helpers shared by the kernels: vector types, 16- and 8-byte
// accesses, the MFMA forms, bf16 / f16 packing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssu {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf2f(uint32_t b16) { return __uint_as_float(b16 << 16); }
__device__ __forceinline__ u32x4 ld16(const void *p) { return *reinterpret_cast<const u32x4 *>(p); }
__device__ __forceinline__ void st16(void *p, u32x4 v) { *reinterpret_cast<u32x4 *>(p) = v; }
__device__ __forceinline__ u32x2 ld8(const void *p) { return *reinterpret_cast<const u32x2 *>(p); }
__device__ __forceinline__ void st8(void *p, u32x2 v) { *reinterpret_cast<u32x2 *>(p) = v; }
// Streaming (non-temporal) forms for data touched once per call whose every
// wave instruction covers whole cache lines (the tiled checkpoint, whose
// chunk u of a row block is 1 KiB contiguous over the wave, the x windows and
// the staged output rows).  Measured on the large-batch step (bf16, batch
// 1024 of 128 heads, one head per wave): its output rows written with plain
// stores took 469 us per step against 450 us with streaming stores.
__device__ __forceinline__ u32x4 ld16_nt(const void *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ void st16_nt(void *p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_f16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Orders this wave's LDS writes before its later LDS reads (no s_barrier).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float softplus_f(float v) { return v > 20.f ? v : log1pf(expf(v)); }

// One of four values for a lane-varying i in [0, 4), taken by value so that
// no register array is indexed at run time (that would go through scratch).
__device__ __forceinline__ float pick4(float v0, float v1, float v2, float v3, int i) {
  return i < 2 ? (i == 0 ? v0 : v1) : (i == 2 ? v2 : v3);
}

__device__ __forceinline__ int ring_pos(int r, int s, int L) {
  int p = r + s;
  return p >= L ? p - L : p;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  _Float16 x = (_Float16)a, y = (_Float16)b;
  return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
}

// Workgroups of a launch go to the 8 XCDs round-robin by ID, and each XCD
// has its own L2.  The one-head-per-wave kernels take their (entry, head tile)
// from xcd_tile, so XCD x runs the contiguous tiles [x per, (x + 1) per): the
// heads of one group, which read the same B and C rows, read them through
// one L2.  The grid is rounded up to a multiple of 8 (tiles >= ntiles idle).
__device__ __forceinline__ int64_t xcd_tile(int64_t id, int64_t ngrid) { return (id & 7) * (ngrid >> 3) + (id >> 3); }
inline unsigned xcd_grid(int64_t ntiles) { return (unsigned)((ntiles + 7) / 8 * 8); }

}  // namespace ssu
