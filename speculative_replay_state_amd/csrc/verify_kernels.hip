// Verification of drafted tokens (ssu_verify).
//
// Two kernels.  verify_sum_kernel, a wave per (entry, piece of 1024 values of
// the vocabulary): the number n of accepted drafts (one lane per draft, a
// ballot), then the sum of the residual r of row n over the piece, in fp64.
// verify_pick_kernel, by the first wave of a workgroup per entry: the piece in which
// the running sum passes u' sum r, the first value in it that does, and the
// bookkeeping.  (The other waves stand by for a residual that is empty, where the
// row itself is summed.)
// verify_row_kernel does both for an entry in one workgroup, where rows are
// short or the entries many.
//
// What bounds them is one read of row n of both distributions, behind the
// drafts' own (dependent) reads.  256 entries of 8 tokens, 131072 bf16 values in
// two distributions: 26.5 us, 5.0 TB/s (32.1 in two launches); 64 entries,
// 100003 fp32 values without draft probabilities (rows no 16 bytes apart):
// 13.0 us (13.5 with those rows read 4 bytes a lane); one entry of 32000: 7.9
// us.  With four pieces a wave of
// verify_sum_kernel 36.7, 14.9 and 10.5 us, with one 32.4, 13.1 and 8.9 (fewer
// waves wait for their drafts); with the verdicts in a kernel of their own
// 31.6, 15.2, 11.9.  An entry whose residual is empty, alone with 131072 fp32
// values: 23 us (94 summed again by one wave); one of the 64 above, with draft
// probabilities, 27 instead of 16 (92); one of the 256 36 instead of 26 (128).
#include "ssu_device.cuh"
#include "verify_internal.h"

#include "../../include/ssu_verify.h"

namespace ssu {

namespace {

constexpr int kLane = kVerifyPiece / 64;  // values of a piece per lane

template <int PT>
__device__ __forceinline__ float prob_at(const uint8_t *row, int i) {
  if constexpr (PT == kPF32) return reinterpret_cast<const float *>(row)[i];
  const uint16_t v = reinterpret_cast<const uint16_t *>(row)[i];
  if constexpr (PT == kPBF16) return bf2f(v);
  return (float)__builtin_bit_cast(_Float16, v);
}

// Eight neighbouring values as they are in memory, 16 bytes at a time from
// wherever the row starts (global loads need no alignment).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <int PT>
struct Eight {
  u32x4 w[PT == kPF32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t *row, int i) {
    const uint8_t *at = row + (int64_t)i * (PT == kPF32 ? 4 : 2);
    w[0] = *reinterpret_cast<const u32x4_any *>(at);
    if constexpr (PT == kPF32) w[1] = *reinterpret_cast<const u32x4_any *>(at + 16);
  }
  __device__ __forceinline__ float value(int k) const {
    if constexpr (PT == kPF32) return __uint_as_float(w[k / 4][k % 4]);
    const uint16_t h = (uint16_t)(w[0][k / 2] >> (16 * (k & 1)));
    return PT == kPBF16 ? bf2f(h) : (float)__builtin_bit_cast(_Float16, h);
  }
};

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
  const int end = v.cu ? v.cu[b + 1] : o.bos + v.T;
  o.T = (int)((uint32_t)end - (uint32_t)o.bos);
  if (o.bos < 0 || end < o.bos || o.T > v.T) {  // (with 0 <= bos <= end the difference cannot wrap)
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

__device__ __forceinline__ float positive(float x) { return x > 0.f ? x : 0.f; }  // NaN: 0

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) x += __shfl_xor(x, s);
  return x;
}

// Sum of r over a piece, in every lane, with every load in flight before the
// first is used.  WIDE (a piece within the vocabulary): 8 neighbours a lane and
// load; else a value a lane, 64 neighbours a load, and past the vocabulary its
// last value, not counted.
template <int PT, bool WIDE>
__device__ __forceinline__ double piece_sum(const KVerify &v, const Verdict &o, bool rejected, int piece, int lane) {
  const int64_t row = (int64_t)o.bos + o.n;
  const bool less = rejected && v.q;  // (without: p is read again, from the cache, and not used)
  const uint8_t *p = v.p + row * v.p_stride, *q = less ? v.q + row * v.q_stride : p;
  const int i0 = piece * kVerifyPiece;
  double sum = 0.0;
  auto add = [&](float a, float b, int i) {
    if (rejected) a -= less ? b : (i == o.draft ? 1.f : 0.f);
    sum += (double)(WIDE || i < v.vocab ? positive(a) : 0.f);
  };
  if constexpr (WIDE) {
    Eight<PT> a[kLane / 8], b[kLane / 8];
#pragma unroll
    for (int k = 0; k < kLane / 8; ++k) {
      a[k].load(p, i0 + k * 512 + lane * 8);
      b[k].load(q, i0 + k * 512 + lane * 8);
    }
#pragma unroll
    for (int k = 0; k < kLane / 8; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) add(a[k].value(e), b[k].value(e), i0 + k * 512 + lane * 8 + e);
  } else {
    float a[kLane], b[kLane];
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      const int i = min(i0 + k * 64 + lane, v.vocab - 1);
      a[k] = prob_at<PT>(p, i);
      b[k] = prob_at<PT>(q, i);
    }
#pragma unroll
    for (int k = 0; k < kLane; ++k) add(a[k], b[k], i0 + k * 64 + lane);
  }
  return wave_sum(sum);
}

template <int PT>
__device__ __forceinline__ double whole_or_part(const KVerify &v, const Verdict &o, bool rejected, int piece, int lane) {
  return (piece + 1) * kVerifyPiece <= v.vocab ? piece_sum<PT, true>(v, o, rejected, piece, lane)
                                               : piece_sum<PT, false>(v, o, rejected, piece, lane);
}

constexpr int kSumWaves = kVerifyGroup / kVerifyPiece;  // waves of a workgroup of verify_sum_kernel
constexpr int kPickWaves = 8;                           // of verify_pick_kernel
constexpr int kRowWaves = 16, kRowPieces = 256;         // of verify_row_kernel; the pieces its LDS holds

// The verdict of an entry in its words of the scratch.
__device__ __forceinline__ Verdict read_verdict(const KVerify &v, const double *ws, int pieces, int b) {
  const int2 w0 = *reinterpret_cast<const int2 *>(ws + pieces), w1 = *reinterpret_cast<const int2 *>(ws + pieces + 1);
  Verdict o;
  o.bos = v.cu ? v.cu[b] : b * v.T;
  o.n = w0.x;
  o.draft = w0.y;
  o.bits = w1.x;
  o.T = w1.y;
  return o;
}
__device__ __forceinline__ void write_verdict(const Verdict &o, double *ws, int pieces) {
  *reinterpret_cast<int2 *>(ws + pieces) = int2{o.n, o.draft};
  *reinterpret_cast<int2 *>(ws + pieces + 1) = int2{o.bits, o.T};
}

template <int PT>
__global__ __launch_bounds__(kSumWaves * 64) void verify_sum_kernel(KVerify v, int pieces) {
  const int lane = threadIdx.x & 63, b = blockIdx.y, piece = blockIdx.x * kSumWaves + (threadIdx.x >> 6);
  if (piece >= pieces) return;
  double *ws = v.ws + (int64_t)b * (pieces + 2);
  const Verdict o = verdict<PT>(v, b, lane);
  if (piece == 0 && lane == 0) write_verdict(o, ws, pieces);
  if (o.T <= 0) return;
  const bool rejected = o.n < o.T - 1 && o.draft >= 0;
  const double sum = whole_or_part<PT>(v, o, rejected, piece, lane);
  if (lane == 0) ws[piece] = sum;
}

// Sums of the lanes up to and with this one.
__device__ __forceinline__ double wave_scan(double x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ int first_lane(uint64_t set) { return (int)__builtin_ctzll(set); }
__device__ __forceinline__ int last_lane(uint64_t set) { return 63 - (int)__builtin_clzll(set); }

// The running sums over an entry's pieces, in LDS or in memory (where they are read
// past the CU's own cache, since the workgroup may have written them itself).
template <bool LDS>
struct Sums {
  double *at;
  int pieces, lane;
  double x, upto, total;  // of this lane's run of neighbouring pieces, up to its end, of all
  __device__ __forceinline__ int first() const { return lane * ((pieces + 63) / 64); }
  __device__ __forceinline__ int end() const { return min(first() + (pieces + 63) / 64, pieces); }
  __device__ __forceinline__ double get(int k) const {
    return LDS ? at[k] : __hip_atomic_load(at + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ void set(int k, double y) const {
    if (lane != 0) return;
    if (LDS)
      at[k] = y;
    else
      __hip_atomic_store(at + k, y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ void add_up() {
    x = 0.0;
    for (int k = first(); k < end(); ++k) x += get(k);
    upto = wave_scan(x, lane);
    total = __shfl(upto, 63);
  }
};

// One wave's pick for entry b; `rejected` is false where an empty residual gave way
// to the row itself.
template <int PT, bool LDS>
__device__ __forceinline__ void pick(const KVerify &v, const Verdict &o, const Sums<LDS> &s, bool rejected, int b, int lane) {
  const double x = s.x, upto = s.upto, total = s.total;
  const int p0 = s.first(), p1 = s.end();
  int bits = o.bits, token = -1;
  if (o.T > 0) {
    if (!(total > 0.0) || total > 1.7e308) {
      bits |= SSU_STATUS_BAD_PROBS;
    } else {
      const float uf = v.uf[b];
      const double want = (double)(uf > 0.f ? uf : 0.f) * total;
      // the run, then the piece in it, whose running sum passes `want`; where
      // rounding leaves none, the last with mass
      const uint64_t over = __ballot(x > 0.0 && upto > want), some = __ballot(x > 0.0);
      const int run = over ? first_lane(over) : last_lane(some);
      int piece = -1;
      double before = upto - x, at = 0.0;  // (in lane `run`)
      for (int k = p0; k < p1; ++k) {
        const double y = s.get(k);
        if (y > 0.0) {
          piece = k;
          at = before;
          if (before + y > want) break;
        }
        before += y;
      }
      piece = __shfl(piece, run);
      at = __shfl(at, run);
      // 16 neighbours a lane
      const int64_t row = (int64_t)o.bos + o.n;
      const uint8_t *p = v.p + row * v.p_stride, *q = rejected && v.q ? v.q + row * v.q_stride : p;
      const int i0 = piece * kVerifyPiece + lane * kLane;
      float r[kLane], less[kLane];
      if ((piece + 1) * kVerifyPiece <= v.vocab) {
        Eight<PT> a[kLane / 8], c[kLane / 8];
#pragma unroll
        for (int k = 0; k < kLane / 8; ++k) {
          a[k].load(p, i0 + 8 * k);
          c[k].load(q, i0 + 8 * k);
        }
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
          r[i] = a[i / 8].value(i % 8);
          less[i] = c[i / 8].value(i % 8);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
          r[i] = prob_at<PT>(p, min(i0 + i, v.vocab - 1));
          less[i] = prob_at<PT>(q, min(i0 + i, v.vocab - 1));
        }
      }
      double mine = 0.0;
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        if (rejected) r[i] -= v.q ? less[i] : (i0 + i == o.draft ? 1.f : 0.f);
        r[i] = i0 + i < v.vocab ? positive(r[i]) : 0.f;
        mine += (double)r[i];
      }
      double sum = at + (wave_scan(mine, lane) - mine);
      int hit = -1, end = -1;
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        sum += (double)r[i];
        if (r[i] > 0.f) {
          end = i;
          if (hit < 0 && sum > want) hit = i;
        }
      }
      const uint64_t hits = __ballot(hit >= 0), ends = __ballot(end >= 0);
      const int from = hits ? first_lane(hits) : last_lane(ends);
      token = piece * kVerifyPiece + from * kLane + __shfl(hits ? hit : end, from);
    }
  }
  const int kept = o.T > 0 ? o.n + 1 : 0;
  if (lane < v.T) {
    int w = -1;
    if (lane + 1 < kept) w = v.tokens[(int64_t)o.bos + lane + 1];
    if (lane + 1 == kept) w = token;
    v.out[(int64_t)b * v.T + lane] = w;
  }
  if (lane == 0) {
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

// Where the residual is empty the row itself is summed, by all waves (they wait for
// the first one's word: with each adding up the sums for itself a row of 2^24 values
// took 133 us, of which 23 were theirs).
template <int PT>
__global__ __launch_bounds__(kPickWaves * 64) void verify_pick_kernel(KVerify v, int pieces) {
  __shared__ int empty;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x;
  double *ws = v.ws + (int64_t)b * (pieces + 2);
  const Verdict o = read_verdict(v, ws, pieces, b);
  bool rejected = o.n < o.T - 1 && o.draft >= 0;  // (the same in every wave)
  Sums<false> s = {ws, pieces, lane, 0.0, 0.0, 0.0};
  if (wave == 0 && o.T > 0) s.add_up();
  if (rejected) {
    if (threadIdx.x == 0) empty = !(s.total > 0.0);
    __syncthreads();
    if (empty) {
      rejected = false;
      for (int k = wave; k < pieces; k += kPickWaves) s.set(k, whole_or_part<PT>(v, o, false, k, lane));
      __threadfence();
      __syncthreads();
      if (wave == 0) s.add_up();
    }
  }
  if (wave == 0) pick<PT, false>(v, o, s, rejected, b, lane);
}

// Both at once: a workgroup per entry, its sums in LDS; every wave forms the
// verdict for itself.  At most kRowPieces pieces (the launch sees to it).
template <int PT>
__global__ __launch_bounds__(kRowWaves * 64) void verify_row_kernel(KVerify v, int pieces) {
  __shared__ double sums[kRowPieces];
  __shared__ int some[kRowWaves];  // whether a wave has found mass
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x;
  const Verdict o = verdict<PT>(v, b, lane);
  bool rejected = o.n < o.T - 1 && o.draft >= 0;
  Sums<true> s = {sums, pieces, lane, 0.0, 0.0, 0.0};
  while (o.T > 0) {
    bool mass = false;
    for (int k = wave; k < pieces; k += kRowWaves) {
      const double y = whole_or_part<PT>(v, o, rejected, k, lane);
      mass |= y > 0.0;
      s.set(k, y);
    }
    if (lane == 0) some[wave] = mass;
    __syncthreads();
    if (!rejected || __ballot(some[lane % kRowWaves]) != 0) break;
    rejected = false;  // an empty residual: the row itself
    __syncthreads();   // (every wave has looked)
  }
  if (wave != 0) return;
  if (o.T > 0) s.add_up();
  pick<PT, true>(v, o, s, rejected, b, lane);
}

template <int PT>
hipError_t verify_pt(const KVerify &v, hipStream_t st) {
  const int pieces = verify_pieces(v.vocab);
  // One launch for short rows (one entry of 4096 values 7.6 us against 10.5, of
  // 40000 bf16 values 10.0 against 10.8, of 65536 12.0 against 10.1), and for
  // entries that fill the card by themselves where the values have two bytes (192
  // rows of 131072 bf16 values 23.0 us against 24.0, 512 48.3 against 55.8; 128
  // rows 22.1 against 18.9; 512 fp32 rows without draft probabilities 60.1
  // against 55.9).
  if (pieces <= 40 || (v.batch >= 192 && PT != kPF32 && pieces <= kRowPieces)) {
    verify_row_kernel<PT><<<dim3((unsigned)v.batch), dim3(kRowWaves * 64), 0, st>>>(v, pieces);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((pieces + kSumWaves - 1) / kSumWaves), (unsigned)v.batch);
  verify_sum_kernel<PT><<<grid, dim3(kSumWaves * 64), 0, st>>>(v, pieces);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  verify_pick_kernel<PT><<<dim3((unsigned)v.batch), dim3(kPickWaves * 64), 0, st>>>(v, pieces);
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
