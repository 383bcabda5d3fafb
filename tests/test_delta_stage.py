"""The staging of prompt chunks (csrc/delta_stage.cuh) run on the host, thread
by thread: what lies in LDS afterwards, and that threads writing one 16-byte
piece all write the same (nothing orders the lanes of a store, or the waves)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <vector>

#include "delta_internal.h"

#ifndef __device__
#define __device__
#endif
#ifndef __forceinline__
#define __forceinline__ inline
#endif
#ifndef __align__
#define __align__(n) __attribute__((aligned(n)))
#endif

namespace ssu {
using std::min;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
struct Range { const char *from, *to; };
static std::vector<Range> readable;
static long bad_reads, conflicts;
static std::map<const char *, u32x4> written;
inline u32x4 ld16(const void *p) {
  const char *at = static_cast<const char *>(p);
  bool ok = (reinterpret_cast<uintptr_t>(p) & 15) == 0, in = false;
  for (const Range &r : readable) in |= at >= r.from && at + 16 <= r.to;
  u32x4 v = {0, 0, 0, 0};
  if (ok && in)
    std::memcpy(&v, p, 16);
  else
    ++bad_reads;
  return v;
}
inline void st16(void *p, u32x4 v) {
  const auto was = written.emplace(static_cast<const char *>(p), v);
  if (!was.second && std::memcmp(&was.first->second, &v, 16) != 0) ++conflicts;
  std::memcpy(p, &v, 16);
}
}  // namespace ssu
#include "delta_stage.cuh"

using namespace ssu;

static uint32_t next_word = 1;
template <class T>
T *fresh(size_t bytes) {  // every word another one
  uint32_t *p = static_cast<uint32_t *>(aligned_alloc(16, (bytes + 15) / 16 * 16));
  for (size_t i = 0; i < bytes / 4; ++i) p[i] = next_word++;
  readable.push_back({reinterpret_cast<char *>(p), reinterpret_cast<char *>(p) + bytes});
  return reinterpret_cast<T *>(p);
}

static int fails;
template <int DK, int COLS, int NP, int NT>
void run(int dv, int len) {
  typedef Chunk<DK, COLS, NP> Buf;
  constexpr int Hk = 2, Hv = 4;
  const int before = 3;  // rows ahead of the sequence
  DPrefill p = {};
  p.Hk = Hk, p.Hv = Hv, p.hpg = 2, p.dk = DK, p.dv = dv;
  p.q_stride = Hk * DK + 8, p.k_stride = Hk * DK, p.v_stride = Hv * dv + 16;
  for (int c0 = 0; c0 < dv; c0 += COLS) {
    readable.clear();
    // only the sequence's rows can be read
    uint16_t *q = fresh<uint16_t>(len * p.q_stride * 2), *k = fresh<uint16_t>(len * p.k_stride * 2), *v = fresh<uint16_t>(len * p.v_stride * 2);
    const int chunks = (len + kChunk - 1) / kChunk;
    uint8_t *rec = fresh<uint8_t>((size_t)chunks * Hv * Buf::kRec);
    p.q = q - before * p.q_stride, p.k = k - before * p.k_stride, p.v = v - before * p.v_stride;
    const Chain n = {before, before + len, 3, c0, chunks};
    const uint8_t *rec0 = rec + (size_t)n.h * Buf::kRec;
    for (int c = 0; c < chunks + 2; ++c) {  // (chunks behind the last are fetched too)
      static Buf buf;
      std::memset(&buf, 0xEE, sizeof buf);
      bad_reads = conflicts = 0;
      written.clear();
      for (int tid = 0; tid < NT; ++tid) {
        Stage<Buf, DK, COLS, NT> st;
        st.fetch(p, n, rec0, c, tid);
        st.store(buf, tid);
      }
      long wrong = 0;
      const int cc = std::min(c, chunks - 1);
      for (int t = 0; t < kChunk; ++t) {
        const int row = std::min(cc * kChunk + t, len - 1);
        wrong += std::memcmp(buf.k + t * Buf::KS, k + row * p.k_stride + DK, DK * 2) != 0;  // (head 3: key head 1)
        wrong += std::memcmp(buf.q + t * Buf::KS, q + row * p.q_stride + DK, DK * 2) != 0;
        const int cols = std::min(COLS, dv - c0);
        wrong += std::memcmp(buf.v + t * Buf::VS, v + row * p.v_stride + 3 * dv + c0, cols * 2) != 0;
      }
      wrong += std::memcmp(buf.rec, rec0 + (size_t)cc * Hv * Buf::kRec, Buf::kRec) != 0;
      for (const auto &w : written) {
        const char *lo = reinterpret_cast<char *>(&buf);
        if (w.first < lo || w.first + 16 > lo + sizeof buf) ++wrong;
      }
      if (bad_reads || conflicts || wrong) {
        ++fails;
        printf("dim_k %d, %d columns, %d parts, %d threads, dim_v %d from %d, %d tokens, chunk %d: %ld reads out of place, "
               "%ld pieces written twice with different values, %ld rows wrong\n", DK, COLS, NP, NT, dv, c0, len, c, bad_reads, conflicts, wrong);
      }
    }
    free(q), free(k), free(v), free(rec);
  }
}

template <int DK, int NP>
void kernels() {
  for (int len : {1, 31, 32, 33, 71}) {
    for (int dv : {16, 48, 64, 80, 128, 144, 256}) {
      run<DK, 16, NP, 4 * 64>(dv, len);   // the chain kernel's helpers
      run<DK, 64, NP, 4 * 64>(dv, len);   // the scan kernel, four waves
      run<DK, 128, NP, 8 * 64>(dv, len);  // and eight
    }
  }
}

int main() {
  kernels<64, 2>(), kernels<64, 3>(), kernels<128, 2>(), kernels<128, 3>();
  printf("%d calls fail\n", fails);
  return fails != 0;
}
"""


def test_every_piece_of_a_chunk_is_staged_once_or_alike(tmp_path):
    clang = next((c for c in ("/opt/rocm/llvm/bin/clang++", shutil.which("amdclang++")) if c and os.path.exists(c)), None)
    if clang is None:
        pytest.skip("no clang++")
    (tmp_path / "stage.cpp").write_text(SOURCE)
    subprocess.run([clang, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "speculative_replay_state_amd", "csrc"), "-I", "/opt/rocm/include",
                    str(tmp_path / "stage.cpp"), "-o", str(tmp_path / "stage")], check=True)
    run = subprocess.run([str(tmp_path / "stage")], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[-2000:]
