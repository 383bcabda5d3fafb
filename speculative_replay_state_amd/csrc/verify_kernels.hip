// Verification of drafted tokens (ssu_verify).
//
// Two kernels.  verify_sum_kernel, a workgroup per (entry, segment of the
// vocabulary): the number n of accepted drafts (one lane per draft, a
// ballot), then the segment's sum of the residual r of row n in fp64.
// verify_pick_kernel, a workgroup per entry: the segment in which the running
// sum passes u' sum r, the first value in it that does, and the bookkeeping.
// What bounds them is one read of row n of both distributions; the second
// kernel reads one segment of it again.
#include "ssu_device.cuh"
#include "verify_internal.h"

#include "../../include/ssu_verify.h"

namespace ssu {

namespace {

constexpr int kT = 256;                       // threads of a workgroup
constexpr int kPer = kVerifySeg / kT;         // values of a segment per thread
constexpr int kWavesV = kT / 64;

template <int PT>
__device__ __forceinline__ float prob_at(const uint8_t *row, int i) {
  if constexpr (PT == kPF32) return reinterpret_cast<const float *>(row)[i];
  const uint16_t v = reinterpret_cast<const uint16_t *>(row)[i];
  if constexpr (PT == kPBF16) return bf2f(v);
  return (float)__builtin_bit_cast(_Float16, v);
}

// 8 values from index i (a multiple of 8) on; 0 past the vocabulary.
template <int PT>
__device__ __forceinline__ void probs8(const uint8_t *row, int i, int vocab, int wide, float (&x)[8]) {
  if (wide && i + 8 <= vocab) {
    if constexpr (PT == kPF32) {
      const f32x4 a = *reinterpret_cast<const f32x4 *>(row + (int64_t)i * 4), b = *reinterpret_cast<const f32x4 *>(row + (int64_t)i * 4 + 16);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = a[r];
        x[4 + r] = b[r];
      }
    } else {
      const u32x4 v = ld16(row + (int64_t)i * 2);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint16_t w = (uint16_t)(v[r / 2] >> (16 * (r & 1)));
        x[r] = PT == kPBF16 ? bf2f(w) : (float)__builtin_bit_cast(_Float16, w);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = i + r < vocab ? prob_at<PT>(row, i + r) : 0.f;
  }
}

struct Verdict {
  int bos, T;   // T < 0: the entry's lengths are not what they have to be
  int n;        // drafts accepted
  int draft;    // the rejected one, -1 if none was (or it is no token)
  int bits;
};

// By one whole wave: lane t tests the draft of row t.
template <int PT>
__device__ __forceinline__ Verdict verdict(const KVerify &v, int b, int lane) {
  Verdict o;
  o.bits = 0;
  o.draft = -1;
  o.n = 0;
  o.bos = v.cu ? v.cu[b] : b * v.T;
  o.T = v.cu ? v.cu[b + 1] - o.bos : v.T;
  if (o.T < 0 || o.T > v.T || o.bos < 0) {
    o.bits = SSU_STATUS_BAD_SEQLEN;
    o.T = -1;
    return o;
  }
  const bool mine = lane < o.T - 1;
  const int64_t row = (int64_t)o.bos + (mine ? lane : 0);
  int d = -1;
  bool ok = false;
  if (mine) {
    d = v.tokens[row + 1];
    if (d >= 0 && d < v.vocab) {
      const double p = prob_at<PT>(v.p + row * v.p_stride, d);
      const double q = v.q ? prob_at<PT>(v.q + row * v.q_stride, d) : 1.f;
      ok = (double)v.u[row] * q < p;
    }
  }
  const uint64_t bad = __ballot(mine && !ok);
  o.n = bad ? __builtin_ctzll(bad) : max(o.T - 1, 0);
  if (bad) {
    d = __shfl(d, o.n);
    if (d >= 0 && d < v.vocab)
      o.draft = d;
    else
      o.bits = SSU_STATUS_BAD_TOKEN;
  }
  return o;
}

// r of values i .. i + 7 of row n
template <int PT>
__device__ __forceinline__ void residual8(const KVerify &v, const Verdict &o, bool rejected, int i, float (&r)[8]) {
  const int64_t row = (int64_t)o.bos + o.n;
  probs8<PT>(v.p + row * v.p_stride, i, v.vocab, v.wide, r);
  if (rejected) {
    if (v.q) {
      float q[8];
      probs8<PT>(v.q + row * v.q_stride, i, v.vocab, v.wide, q);
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] -= q[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] -= i + k == o.draft ? 1.f : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = r[k] > 0.f ? r[k] : 0.f;  // NaN: 0
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) x += __shfl_xor(x, s);
  return x;
}

template <int PT>
__global__ __launch_bounds__(kT) void verify_sum_kernel(KVerify v) {
  __shared__ double part[kWavesV];
  const int tid = threadIdx.x, lane = tid & 63, b = blockIdx.y, seg = blockIdx.x;
  const Verdict o = verdict<PT>(v, b, lane);
  if (o.T <= 0) return;
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kPer / 8; ++k) {
    float r[8];
    residual8<PT>(v, o, o.n < o.T - 1 && o.draft >= 0, seg * kVerifySeg + (k * kT + tid) * 8, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (double)r[i];
  }
  sum = wave_sum(sum);
  if (lane == 0) part[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) v.ws[(int64_t)b * gridDim.x + seg] = part[0] + part[1] + part[2] + part[3];
}

// Sums of the threads before this one, and of all, over the workgroup.
__device__ __forceinline__ double block_scan(double x, int tid, double *part, double *total) {
  const int lane = tid & 63, wave = tid >> 6;
  double s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();  // `part` may still be read from the scan before
  if (lane == 63) part[wave] = s;
  __syncthreads();
  double before = 0.0, all = 0.0;
#pragma unroll
  for (int w = 0; w < kWavesV; ++w) {
    if (w < wave) before += part[w];
    all += part[w];
  }
  *total = all;
  return before + (s - x);
}

// The smallest (SMALL) or largest of the threads' values.
template <bool SMALL>
__device__ __forceinline__ int block_pick(int x, int tid, int *part) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const int y = __shfl_xor(x, s);
    x = SMALL ? min(x, y) : max(x, y);
  }
  __syncthreads();
  if ((tid & 63) == 0) part[tid >> 6] = x;
  __syncthreads();
  x = part[0];
#pragma unroll
  for (int w = 1; w < kWavesV; ++w) x = SMALL ? min(x, part[w]) : max(x, part[w]);
  return x;
}

// Sum of r over the row, from scratch (only where the residual is empty).
template <int PT>
__device__ double row_mass(const KVerify &v, const Verdict &o, int tid, double *part, double *seg_sum, int nseg) {
  for (int s = 0; s < nseg; ++s) {
    double x = 0.0, all;
    for (int k = 0; k < kPer / 8; ++k) {
      float r[8];
      residual8<PT>(v, o, false, s * kVerifySeg + (k * kT + tid) * 8, r);
      for (int i = 0; i < 8; ++i) x += (double)r[i];
    }
    block_scan(x, tid, part, &all);
    if (tid == 0) seg_sum[s] = all;
  }
  __threadfence_block();
  __syncthreads();
  double sum = 0.0;
  for (int s = tid; s < nseg; s += kT) sum += seg_sum[s];
  double all;
  block_scan(sum, tid, part, &all);
  return all;
}

template <int PT>
__global__ __launch_bounds__(kT) void verify_pick_kernel(KVerify v, int nseg) {
  __shared__ double part[kWavesV];
  __shared__ int ipart[kWavesV];
  __shared__ double s_before;
  __shared__ int s_seg;
  const int tid = threadIdx.x, lane = tid & 63, b = blockIdx.x;
  const Verdict o = verdict<PT>(v, b, lane);
  int bits = o.bits, token = -1;
  if (o.T > 0) {
    double *sums = v.ws + (int64_t)b * nseg;
    bool rejected = o.n < o.T - 1 && o.draft >= 0;
    double x = 0.0, total;
    for (int s = tid; s < nseg; s += kT) x += sums[s];
    block_scan(x, tid, part, &total);
    if (!(total > 0.0) && rejected) {
      rejected = false;
      total = row_mass<PT>(v, o, tid, part, sums, nseg);
    }
    if (!(total > 0.0) || total > 1.7e308) {
      bits |= SSU_STATUS_BAD_PROBS;
    } else {
      const float uf = v.uf[b];
      const double want = (double)(uf > 0.f ? uf : 0.f) * total;
      // the first segment whose running sum passes `want`, else the last with mass
      if (tid == 0) s_seg = -1;
      int found = nseg;
      double base = 0.0;
      for (int s0 = 0; s0 < nseg && found == nseg; s0 += kT) {
        const int s = s0 + tid;
        const double y = s < nseg ? sums[s] : 0.0;
        double all;
        const double before = base + block_scan(y, tid, part, &all);
        found = block_pick<true>(y > 0.0 && before + y > want ? s : nseg, tid, ipart);
        const int l = block_pick<false>(y > 0.0 ? s : -1, tid, ipart);
        if (s == (found < nseg ? found : l) && y > 0.0) {
          s_seg = s;
          s_before = before;
        }
        base += all;
      }
      __syncthreads();
      const int seg = s_seg;
      const double start = s_before;
      // values in order: thread t holds 16 neighbours
      float r[kPer];
      double sum = 0.0;
#pragma unroll
      for (int k = 0; k < kPer / 8; ++k) {
        float y[8];
        residual8<PT>(v, o, rejected, seg * kVerifySeg + tid * kPer + k * 8, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[8 * k + i] = y[i];
          sum += (double)y[i];
        }
      }
      double all;
      double run = start + block_scan(sum, tid, part, &all);
      int hit = v.vocab, end = -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = seg * kVerifySeg + tid * kPer + i;
        run += (double)r[i];
        if (r[i] > 0.f) {
          end = at;
          if (run > want && hit == v.vocab) hit = at;
        }
      }
      hit = block_pick<true>(hit, tid, ipart);
      end = block_pick<false>(end, tid, ipart);
      token = hit < v.vocab ? hit : end;
    }
  }
  const int kept = o.T > 0 ? o.n + 1 : 0;
  if (tid < v.T) {
    int w = -1;
    if (tid + 1 < kept) w = v.tokens[(int64_t)o.bos + tid + 1];
    if (tid + 1 == kept) w = token;
    v.out[(int64_t)b * v.T + tid] = w;
  }
  if (tid == 0) {
    v.accepted[b] = kept;
    if (v.next_live) {
      const int left = v.live[b] - (v.fold ? v.fold[b] : 0) + kept;
      const int fold = left + v.reserve > v.ring_len ? left : 0;
      v.next_live[b] = left;
      if (v.next_fold) v.next_fold[b] = fold;
      if (v.next_left) v.next_left[b] = left - fold;
    }
    if (bits && v.status) atomicOr(v.status, bits);
  }
}

template <int PT>
hipError_t verify_pt(const KVerify &v, hipStream_t st) {
  const int nseg = verify_segments(v.vocab);
  verify_sum_kernel<PT><<<dim3((unsigned)nseg, (unsigned)v.batch), dim3(kT), 0, st>>>(v);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  verify_pick_kernel<PT><<<dim3((unsigned)v.batch), dim3(kT), 0, st>>>(v, nseg);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const KVerify &v, int prob_type, hipStream_t st) {
  switch (prob_type) {
    case kPF32: return verify_pt<kPF32>(v, st);
    case kPBF16: return verify_pt<kPBF16>(v, st);
    default: return verify_pt<kPF16>(v, st);
  }
}

}  // namespace ssu
