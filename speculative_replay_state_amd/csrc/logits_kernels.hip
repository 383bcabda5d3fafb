// Token histories (ssu_history_count) and logits (ssu_logits).
//
// A row's values go through registers 8 neighbours a lane.  Few of them are
// special, in the history, among the drafts or biased: a workgroup marks those of its
// range in a bitmap in LDS, numbers them by the set bits before them, and a thread
// each forms their x (a load of the logit and of the count, all at once) into LDS,
// from where the lane that holds the value takes it.
#include "logits_internal.h"
#include "ssu_device.cuh"

#include "../../include/ssu_logits.h"

#include <float.h>

namespace ssu {

namespace {

// ---------------------------------------------------------------------------
// histories
// ---------------------------------------------------------------------------

// A workgroup per entry.  A word of `counts` whose bit was not set yet is
// emptied by the one thread that sets the bit, then all tokens are added:
// nothing but the bits has to be cleared for a new request.
template <int NT>
__global__ __launch_bounds__(NT) void count_kernel(KHistory h, KCount c) {
  const int b = blockIdx.x, tid = threadIdx.x, slot = c.slot_idx[b];
  if (slot <= 0 || slot >= h.num_slots) return;
  int64_t first = (int64_t)b * c.T;
  int n = c.T;
  bool ok;
  if (c.cu) {
    const int b0 = c.cu[b], b1 = c.cu[b + 1];
    ok = b0 >= 0 && b0 <= b1 && b1 <= c.rows;
    first = b0;
    n = b1 - b0;
  } else {
    if (c.num) n = c.num[b];
    ok = n >= 0 && n <= c.T;
  }
  if (!ok) {
    if (tid == 0 && h.status) atomicOr(h.status, SSU_STATUS_BAD_SEQLEN);
    return;
  }
  uint32_t *seen = h.seen + (int64_t)slot * h.seen_stride;
  int32_t *counts = h.counts + (int64_t)slot * h.counts_stride;
  const int32_t *tokens = c.tokens + first;
  if (c.reset) {
    for (int w = tid; w < h.words; w += NT) seen[w] = 0;
    __threadfence();
    __syncthreads();
  }
  constexpr int U = 4;
  bool bad = false;
  for (int i = tid; i < n; i += NT * U) {
    int tok[U];
    uint32_t old[U];
#pragma unroll
    for (int u = 0; u < U; ++u) tok[u] = i + u * NT < n ? tokens[i + u * NT] : -2;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = tok[u] >= 0 && tok[u] < h.vocab;
      bad |= !in && tok[u] != -2;
      bad |= tok[u] == -2 && i + u * NT < n;
      old[u] = in ? atomicOr(seen + (tok[u] >> 5), 1u << (tok[u] & 31)) : ~0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (!((old[u] >> (tok[u] & 31)) & 1)) counts[tok[u]] = 0;
  }
  if (bad && h.status) atomicOr(h.status, SSU_STATUS_BAD_TOKEN);
  __threadfence();
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const int tok = tokens[i];
    if (tok < 0 || tok >= h.vocab) continue;
    if (c.prompt)
      atomicOr(counts + tok, 1);
    else
      atomicAdd(counts + tok, 2);
  }
}

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------

constexpr int logit_size(int T) { return T == kLF32 ? 4 : 2; }

template <int IT>
__device__ __forceinline__ float logit_at(const uint8_t *row, int i) {
  if constexpr (IT == kLF32) return reinterpret_cast<const float *>(row)[i];
  const uint16_t v = reinterpret_cast<const uint16_t *>(row)[i];
  if constexpr (IT == kLBF16) return bf2f(v);
  return (float)__builtin_bit_cast(_Float16, v);
}

// Eight neighbouring values as they are in memory, 16 bytes at a time from
// wherever the row starts (global accesses need no alignment).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <int IT>
struct Eight {
  u32x4 w[IT == kLF32 ? 2 : 1];
  __device__ __forceinline__ float value(int k) const {
    if constexpr (IT == kLF32) return __uint_as_float(w[k / 4][k % 4]);
    const uint16_t h = (uint16_t)(w[0][k / 2] >> (16 * (k & 1)));
    return IT == kLBF16 ? bf2f(h) : (float)__builtin_bit_cast(_Float16, h);
  }
  // values i .. i + 7 of a row of n; past its end the last one, again
  __device__ __forceinline__ void load(const uint8_t *row, int i, int n) {
    constexpr int S = logit_size(IT);
    if (i + 8 <= n) {
      const uint8_t *at = row + (int64_t)i * S;
      w[0] = *reinterpret_cast<const u32x4_any *>(at);
      if constexpr (IT == kLF32) w[1] = *reinterpret_cast<const u32x4_any *>(at + 16);
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = min(i + k, n - 1);
      if constexpr (IT == kLF32) {
        w[k / 4][k % 4] = reinterpret_cast<const uint32_t *>(row)[at];
      } else {
        const uint32_t v = reinterpret_cast<const uint16_t *>(row)[at];
        w[0][k / 2] = k & 1 ? (w[0][k / 2] & 0xFFFFu) | (v << 16) : v;
      }
    }
  }
};

template <int OT>
__device__ __forceinline__ void store8(uint8_t *row, int i, int n, const float (&v)[8]) {
  uint8_t *at = row + (int64_t)i * logit_size(OT);
  if (i + 8 <= n) {
    if constexpr (OT == kLF32) {
      u32x4 a, b;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = __float_as_uint(v[k]);
        b[k] = __float_as_uint(v[4 + k]);
      }
      *reinterpret_cast<u32x4_any *>(at) = a;
      *reinterpret_cast<u32x4_any *>(at + 16) = b;
    } else {
      u32x4 a;
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = OT == kLBF16 ? pack_bf16(v[2 * k], v[2 * k + 1]) : pack_f16(v[2 * k], v[2 * k + 1]);
      *reinterpret_cast<u32x4_any *>(at) = a;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (i + k >= n) break;
    if constexpr (OT == kLF32)
      reinterpret_cast<float *>(at)[k] = v[k];
    else
      reinterpret_cast<uint16_t *>(at)[k] = (uint16_t)(OT == kLBF16 ? pack_bf16(v[k], 0.f) : pack_f16(v[k], 0.f));
  }
}

// What a workgroup needs of its row.
struct Row {
  int64_t row;
  const uint8_t *in;
  const uint32_t *seen;   // NULL: no history
  const int32_t *counts;
  const int32_t *drafts;  // nd tokens fed up to this row
  int nd;
  const int32_t *bias_tok;
  const float *bias_val;
  int nb;
  const uint8_t *mask;    // NULL: all
  float rep, freq, pres, temperature;
};

// Row t of entry b; false where there is none.  `report`: bits are set.
__device__ __forceinline__ bool find_row(const KHistory &h, const KLogits &l, int b, int t, bool report, Row &r) {
  int b0 = b * l.T, n = l.T;
  if (l.cu) {
    const int b1 = l.cu[b + 1];
    b0 = l.cu[b];
    n = b0 >= 0 && b0 <= b1 && b1 <= l.rows ? b1 - b0 : -1;
    if (n > l.T) n = -1;
    if (n < 0 && t == 0 && report && l.status) atomicOr(l.status, SSU_STATUS_BAD_SEQLEN);
  }
  if (t >= n) return false;
  r.row = (int64_t)b0 + t;
  r.in = l.in + r.row * l.in_stride;
  r.seen = nullptr;
  r.counts = nullptr;
  r.drafts = nullptr;
  r.nd = 0;
  if (h.counts) {
    const int slot = l.slot_idx ? l.slot_idx[b] : 0;
    if (slot > 0 && slot < h.num_slots) {
      r.seen = h.seen + (int64_t)slot * h.seen_stride;
      r.counts = h.counts + (int64_t)slot * h.counts_stride;
    }
    if (l.tokens) {
      r.drafts = l.tokens + b0 + 1;
      r.nd = t;
    }
  }
  r.nb = 0;
  r.bias_tok = l.bias_tok;
  r.bias_val = l.bias_val;
  if (l.bias_off) {
    const int o0 = l.bias_off[b], o1 = l.bias_off[b + 1];
    if (o0 >= 0 && o0 <= o1 && o1 <= l.bias_count) {
      r.bias_tok += o0;
      r.bias_val += o0;
      r.nb = o1 - o0;
    } else if (report && t == 0 && l.status) {
      atomicOr(l.status, SSU_STATUS_BAD_BIAS);
    }
  }
  r.mask = l.mask ? reinterpret_cast<const uint8_t *>(l.mask + r.row * l.mask_stride) : nullptr;
  r.rep = l.repetition ? l.repetition[b] : 1.f;
  r.freq = l.frequency ? l.frequency[b] : 0.f;
  r.pres = l.presence ? l.presence[b] : 0.f;
  r.temperature = l.temperature ? l.temperature[b] : 1.f;
  return true;
}

// x of a special token: its logit, the bias (if it has one), whether it was there and how many times.
__device__ __forceinline__ float special_x(const Row &r, float x, bool biased, float bias, bool was, int n) {
  if (biased) x = x + bias;
  if (was) {
    x = x > 0.f ? x / r.rep : x * r.rep;
    x = x - (r.freq * (float)n + (n > 0 ? r.pres : 0.f));
  }
  return x;
}

// The special tokens of the values [i0, i0 + 32 * words) of a row.
template <int NT, int WORDS, int CAP>
struct Special {
  uint32_t bits[WORDS];
  uint16_t rank[WORDS];    // set bits before the word
  uint32_t info[CAP];      // by rank: 256 (its last bias + 1) + its drafts
  float x[CAP];            // by rank
  int sums[NT / 64];

  __device__ __forceinline__ int at(int i) const {  // rank of value i of the range
    return rank[i >> 5] + __builtin_popcount(bits[i >> 5] & ((1u << (i & 31)) - 1u));
  }

  // By the whole workgroup; the number of special tokens (more than CAP: only their bits are there).
  template <int IT>
  __device__ __forceinline__ int build(const Row &r, int i0, int words, int vocab, int tid) {
    if (!r.seen && r.nd == 0 && r.nb == 0) return 0;
    const int end = min(i0 + 32 * words, vocab);
    for (int w = tid; w < words; w += NT) {
      uint32_t v = r.seen ? r.seen[(i0 >> 5) + w] : 0u;
      const int left = vocab - i0 - 32 * w;
      if (left < 32) v &= (1u << left) - 1u;  // (left > 0: the words are the vocabulary's)
      bits[w] = v;
    }
    __syncthreads();
    if (r.nd > 0 || r.nb > 0) {
      for (int j = tid; j < r.nd; j += NT) {
        const int k = r.drafts[j];
        if (k >= i0 && k < end) atomicOr(&bits[(k - i0) >> 5], 1u << (k & 31));
      }
      for (int j = tid; j < r.nb; j += NT) {
        const int k = r.bias_tok[j];
        if (k >= i0 && k < end) atomicOr(&bits[(k - i0) >> 5], 1u << (k & 31));
      }
      __syncthreads();
    }
    // set bits before each word: a thread takes neighbouring words
    const int lane = tid & 63, each = (words + NT - 1) / NT, w0 = min(tid * each, words), w1 = min(w0 + each, words);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __builtin_popcount(bits[w]);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 63) sums[tid >> 6] = upto;
    __syncthreads();
    int before = upto - mine, total = 0;
#pragma unroll
    for (int k = 0; k < NT / 64; ++k) {
      if (k < (tid >> 6)) before += sums[k];
      total += sums[k];
    }
    if (total == 0 || (CAP < 32 * WORDS && total > CAP)) return total;
    for (int w = w0; w < w1; ++w) {
      rank[w] = (uint16_t)before;
      for (uint32_t v = bits[w]; v; v &= v - 1) {
        x[before] = __int_as_float(32 * w + __builtin_ctz(v));
        info[before++] = 0;
      }
    }
    __syncthreads();
    if (r.nb > 0) {
      for (int j = tid; j < r.nb; j += NT) {
        const int k = r.bias_tok[j];
        if (k >= i0 && k < end) atomicMax(&info[at(k - i0)], (uint32_t)(j + 1) << 8);
      }
      __syncthreads();
    }
    if (r.nd > 0) {
      for (int j = tid; j < r.nd; j += NT) {
        const int k = r.drafts[j];
        if (k >= i0 && k < end) atomicAdd(&info[at(k - i0)], 1u);
      }
      __syncthreads();
    }
    for (int j = tid; j < total; j += NT) {
      const int i = i0 + __float_as_int(x[j]);
      const uint32_t f = info[j];
      const float v = logit_at<IT>(r.in, i);
      int n = (int)(f & 255u);
      bool was = n > 0;
      if (r.seen && (r.seen[i >> 5] >> (i & 31)) & 1u) {
        was = true;
        n += r.counts[i] >> 1;
      }
      x[j] = special_x(r, v, f >> 8, f >> 8 ? r.bias_val[(f >> 8) - 1] : 0.f, was, n);
    }
    __syncthreads();
    return total;
  }

  // x of the values i .. i + 7 of the row (i0 the range's start), -inf where there is none.
  template <int IT>
  __device__ __forceinline__ void values(const Row &r, const Eight<IT> &e, int total, int i0, int i, int vocab, float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = e.value(k);
    if (total > 0) {
      const int o = i - i0;
      const uint32_t word = bits[o >> 5], byte = (word >> (o & 31)) & 255u;
      if (byte) {
        if (CAP >= 32 * WORDS || total <= CAP) {
          int j = at(o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if ((byte >> k) & 1u) v[k] = x[j++];
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if ((byte >> k) & 1u) v[k] = slow(r, v[k], i + k);
        }
      }
    }
    uint32_t allowed = r.mask && i < vocab ? r.mask[i >> 3] : 255u;
    if (i + 8 > vocab) allowed &= i < vocab ? (1u << (vocab - i)) - 1u : 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (allowed >> k) & 1u && v[k] == v[k] ? v[k] : -INFINITY;
  }

  // Where the range holds more special tokens than LDS has room for.
  static __device__ __forceinline__ float slow(const Row &r, float x, int i) {
    int bias = -1, n = 0;
    for (int j = 0; j < r.nb; ++j)
      if (r.bias_tok[j] == i) bias = j;
    for (int j = 0; j < r.nd; ++j) n += r.drafts[j] == i;
    bool was = n > 0;
    if (r.seen && (r.seen[i >> 5] >> (i & 31)) & 1u) {
      was = true;
      n += r.counts[i] >> 1;
    }
    return special_x(r, x, bias >= 0, bias >= 0 ? r.bias_val[bias] : 0.f, was, n);
  }
};

// The largest x and sum of exp((x - m) / temperature), or for the greedy
// choice the index of the first x = m (in the bits of s).
struct Stat {
  float m, s;
};
__device__ __forceinline__ float decay_to(float m, float M, float k) {
  return __builtin_amdgcn_exp2f((m - fmaxf(M, -FLT_MAX)) * k);
}
__device__ __forceinline__ Stat join(Stat a, Stat b, float k, bool greedy) {
  if (greedy) {
    const bool first = a.m > b.m || (a.m == b.m && __float_as_uint(a.s) <= __float_as_uint(b.s));
    return Stat{first ? a.m : b.m, first ? a.s : b.s};
  }
  Stat o;
  o.m = fmaxf(a.m, b.m);
  o.s = a.s * decay_to(a.m, o.m, k) + b.s * decay_to(b.m, o.m, k);
  return o;
}
// log2(e) / temperature, finite and positive: (x - m) times it is 0 at x = m and -inf at x = -inf
__device__ __forceinline__ float slope(float temperature) {
  return fminf(fmaxf(1.4426950408889634f / temperature, FLT_MIN), FLT_MAX);
}
__device__ __forceinline__ bool is_greedy(float temperature) { return !(temperature > 0.f); }

__device__ __forceinline__ void add8(Stat &o, float (&v)[8], int i, float k, bool greedy) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fminf(v[e], FLT_MAX);
  if (greedy) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (v[e] > o.m) {
        o.m = v[e];
        o.s = __uint_as_float((uint32_t)(i + e));
      }
    return;
  }
  float m = o.m;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, v[e]);
  const float M = fmaxf(m, -FLT_MAX);
  float s = o.s * __builtin_amdgcn_exp2f((o.m - M) * k);
#pragma unroll
  for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((v[e] - M) * k);
  o.m = m;
  o.s = s;
}
__device__ __forceinline__ Stat no_stat(bool greedy) { return Stat{-INFINITY, greedy ? __uint_as_float(~0u) : 0.f}; }

// In every thread.
template <int NT>
__device__ __forceinline__ Stat block_join(Stat s, Stat *lds, int tid, float k, bool greedy) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s = join(s, Stat{__shfl_xor(s.m, d), __shfl_xor(s.s, d)}, k, greedy);
  __syncthreads();
  if ((tid & 63) == 0) lds[tid >> 6] = s;
  __syncthreads();
  Stat o = lds[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) o = join(o, lds[w], k, greedy);
  return o;
}

// The probabilities of eight values of a row whose statistics are s.
__device__ __forceinline__ void probs8(float (&v)[8], int i, Stat s, float inv, float k, bool greedy) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (greedy)
      v[e] = (uint32_t)(i + e) == __float_as_uint(s.s) ? 1.f : 0.f;
    else
      v[e] = __builtin_amdgcn_exp2f((fminf(v[e], FLT_MAX) - fmaxf(s.m, -FLT_MAX)) * k) * inv;
  }
}
__device__ __forceinline__ float inverse(Stat s) { return s.m > -INFINITY ? 1.f / s.s : 0.f; }

constexpr int kPieceThreads = 256;

// MODE 0: statistics of a piece of a row into the workspace.  1: the probabilities of the
// piece from them.  2: the piece's x / temperature.
template <int IT, int OT, int G, int MODE>
__global__ __launch_bounds__(kPieceThreads) void logits_piece_kernel(KHistory h, KLogits l, int pieces) {
  constexpr int NT = kPieceThreads, PIECE = NT * 8 * G;
  typedef Special<NT, PIECE / 32, PIECE> Sp;
  __shared__ Sp sp;
  __shared__ Stat red[NT / 64];
  const int tid = threadIdx.x, piece = blockIdx.x, b = blockIdx.y / l.T, t = blockIdx.y - b * l.T;
  Row r;
  if (!find_row(h, l, b, t, piece == 0 && tid == 0 && MODE != 1, r)) return;
  const int i0 = piece * PIECE;
  Eight<IT> e[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int i = i0 + (g * NT + tid) * 8;
    if (i < l.vocab) e[g].load(r.in, i, l.vocab);
  }
  const bool greedy = is_greedy(r.temperature);
  const float k = slope(r.temperature);
  float2 *ws = l.ws + (int64_t)blockIdx.y * pieces;
  Stat s = no_stat(greedy);
  if constexpr (MODE == 1) {
    for (int j = tid; j < pieces; j += NT) {
      const float2 w = ws[j];
      s = join(s, Stat{w.x, w.y}, k, greedy);
    }
  }
  const int total = sp.template build<IT>(r, i0, (min(PIECE, l.vocab - i0) + 31) / 32, l.vocab, tid);
  if constexpr (MODE == 1) s = block_join<NT>(s, red, tid, k, greedy);
  const float inv = inverse(s);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int i = i0 + (g * NT + tid) * 8;
    if (i >= l.vocab) continue;
    float v[8];
    sp.template values<IT>(r, e[g], total, i0, i, l.vocab, v);
    if constexpr (MODE == 0) {
      add8(s, v, i, k, greedy);
    } else {
      if constexpr (MODE == 1) {
        probs8(v, i, s, inv, k, greedy);
      } else if (!greedy) {
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = v[x] / r.temperature;
      }
      store8<OT>(l.out + r.row * l.out_stride, i, l.vocab, v);
    }
  }
  if constexpr (MODE == 0) {
    s = block_join<NT>(s, red, tid, k, greedy);
    if (tid == 0) ws[piece] = float2{s.m, s.s};
  }
  if (MODE == 1 && piece == 0 && tid == 0 && l.status && !(s.m > -INFINITY)) atomicOr(l.status, SSU_STATUS_EMPTY_ROW);
  if (MODE != 1 && piece == 0 && l.status && r.nb > 0 && t == 0) {
    bool bad = false;
    for (int j = tid; j < r.nb; j += NT) bad |= r.bias_tok[j] < 0 || r.bias_tok[j] >= l.vocab;
    if (bad) atomicOr(l.status, SSU_STATUS_BAD_BIAS);
  }
}

template <int IT, int OT>
hipError_t logits_t(const KHistory &h, const KLogits &l, bool softmax, hipStream_t st) {
  constexpr int G = 1;
  const int pieces = (l.vocab + kPieceThreads * 8 * G - 1) / (kPieceThreads * 8 * G);
  const dim3 grid((unsigned)pieces, (unsigned)(l.batch * l.T)), block(kPieceThreads);
  if (!softmax) {
    logits_piece_kernel<IT, OT, G, 2><<<grid, block, 0, st>>>(h, l, pieces);
    return hipGetLastError();
  }
  logits_piece_kernel<IT, kLF32, G, 0><<<grid, block, 0, st>>>(h, l, pieces);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  logits_piece_kernel<IT, OT, G, 1><<<grid, block, 0, st>>>(h, l, pieces);
  return hipGetLastError();
}

template <int IT>
hipError_t logits_it(const KHistory &h, const KLogits &l, int out_type, bool softmax, hipStream_t st) {
  switch (out_type) {
    case kLF32: return logits_t<IT, kLF32>(h, l, softmax, st);
    case kLBF16: return logits_t<IT, kLBF16>(h, l, softmax, st);
    default: return logits_t<IT, kLF16>(h, l, softmax, st);
  }
}

}  // namespace

hipError_t launch_count(const KHistory &h, const KCount &c, hipStream_t st) {
  if (!c.reset && !c.cu && c.T <= 64)
    count_kernel<64><<<dim3((unsigned)c.batch), dim3(64), 0, st>>>(h, c);
  else
    count_kernel<1024><<<dim3((unsigned)c.batch), dim3(1024), 0, st>>>(h, c);
  return hipGetLastError();
}

hipError_t launch_logits(const KHistory &h, const KLogits &l, int in_type, int out_type, bool softmax, hipStream_t st) {
  switch (in_type) {
    case kLF32: return logits_it<kLF32>(h, l, out_type, softmax, st);
    case kLBF16: return logits_it<kLBF16>(h, l, out_type, softmax, st);
    default: return logits_it<kLF16>(h, l, out_type, softmax, st);
  }
}

}  // namespace ssu
