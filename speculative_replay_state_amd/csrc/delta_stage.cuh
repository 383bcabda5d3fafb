// A prompt chunk's way from memory to LDS: what the waves of a chain share and
// the registers that bring it there.  Included after the vector type and the
// 16-byte accesses it uses (ssu_device.cuh), with nothing else of the device in
// it: a test runs it on the host, every thread and every word.
#pragma once

#include <stdint.h>

#include "delta_internal.h"

namespace ssu {

// 16-byte pieces of a chunk that NT threads stage, per thread.
constexpr int pieces(int n, int NT) { return (n + NT - 1) / NT; }

// What the waves of a chain share of a chunk.  (Rows that avoid the bank
// conflicts of the transposed reads, 16 banks apart instead of 4, halve those
// conflicts and change no time: 622 us either way for 8 sequences of 2048 to 4096
// tokens, 64 heads of dim 128.)
template <int DK, int COLS, int NP>
struct Chunk {
  static constexpr int kRec = rec_bytes(NP);
  static constexpr int KS = DK + 8, VS = COLS + 8;  // row strides: 16 rows start in different banks
  __align__(16) uint16_t k[kChunk * KS], q[kChunk * KS], v[kChunk * VS];
  __align__(16) uint8_t rec[kRec];
  __device__ __forceinline__ const float *factors() const { return reinterpret_cast<const float *>(rec + rec_t(NP)); }
};

// One sequence's chunks of a head's columns c0 .. c0 + COLS - 1.
struct Chain {
  int b0, b1, h, c0, chunks;
};

// A chunk on its way from memory to LDS through the registers of NT threads.
// Every load is unconditional, so that the waits of a loop around them count
// exactly: behind the sequence's end (and the last chunk) they repeat its last
// row (and chunk), whose gates in the record are 0, and columns behind dim_v
// repeat the first ones.
template <class Buf, int DK, int COLS, int NT>
struct Stage {
  // piece i of a thread, of n in all: a thread without one of its own takes the
  // last, in the load as in the store, so that all who write it write the same
  static __device__ __forceinline__ int piece(int i, int tid, int n) { return min(i * NT + tid, n - 1); }
  static constexpr int NK = kChunk * DK / 8, NV = kChunk * COLS / 8, NR = Buf::kRec / 16;
  static constexpr int PK = pieces(NK, NT), PV = pieces(NV, NT), PR = pieces(NR, NT);
  u32x4 k[PK], q[PK], v[PV], r[PR];

  __device__ __forceinline__ void fetch(const DPrefill &p, const Chain &n, const uint8_t *rec0, int c, int tid) {
    c = min(c, n.chunks - 1);
    const int last = min(kChunk, n.b1 - n.b0 - c * kChunk) - 1;
    // uniform bases and 32-bit byte offsets of the lanes
    const int64_t row = n.b0 + c * kChunk;
    const int hk = n.h / p.hpg, ks = (int)p.k_stride * 2, qs = (int)p.q_stride * 2, vs = (int)p.v_stride * 2;
    const char *kc = reinterpret_cast<const char *>(p.k + row * p.k_stride + hk * DK);
    const char *qc = reinterpret_cast<const char *>(p.q + row * p.q_stride + hk * DK);
    const char *vc = reinterpret_cast<const char *>(p.v + row * p.v_stride + n.h * p.dv + n.c0);
    const uint8_t *rec = rec0 + (int64_t)c * p.Hv * Buf::kRec;
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const int at = piece(i, tid, NK), t = min(at / (DK / 8), last), ch = at % (DK / 8);
      k[i] = ld16(kc + (uint32_t)(t * ks + ch * 16));
      q[i] = ld16(qc + (uint32_t)(t * qs + ch * 16));
    }
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      const int at = piece(i, tid, NV), t = min(at / (COLS / 8), last), ch = at % (COLS / 8);
      v[i] = ld16(vc + (uint32_t)(t * vs + (n.c0 + ch * 8 < p.dv ? ch * 16 : 0)));
    }
#pragma unroll
    for (int i = 0; i < PR; ++i) r[i] = ld16(rec + (uint32_t)(piece(i, tid, NR) * 16));
  }

  __device__ __forceinline__ void store(Buf &o, int tid) const {
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const int at = piece(i, tid, NK), t = at / (DK / 8), ch = at % (DK / 8);
      st16(o.k + t * Buf::KS + ch * 8, k[i]);
      st16(o.q + t * Buf::KS + ch * 8, q[i]);
    }
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      const int at = piece(i, tid, NV), t = at / (COLS / 8), ch = at % (COLS / 8);
      st16(o.v + t * Buf::VS + ch * 8, v[i]);
    }
#pragma unroll
    for (int i = 0; i < PR; ++i) st16(o.rec + piece(i, tid, NR) * 16, r[i]);
  }
};

}  // namespace ssu
