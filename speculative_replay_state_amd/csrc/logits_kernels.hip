// Token histories (ssu_history_count) and logits (ssu_logits).
//
// The softmax takes every value twice, for the largest x and the sum of exp((x - m) /
// temperature), and for the probabilities; memory bounds it from some hundred rows on.
// The first values of a row stay in registers between the two; the others come again, from
// the last cache where the rows under way are more than an L2 holds (64 of them an XCD: of
// 131072 bf16 values 16 MiB for 4, and 995 MiB are read for 442 of logits and masks).  They
// go through registers 8 neighbours a lane, with a byte of a bitmap in LDS that says
// which of them are not taken as they are: these become NaN, which counts for nothing
// (a maximum passes over it, the exponential's own bounds of 0 and 1 make it 0; so a
// value costs some ten instructions in each of the two).  Those in the history, among
// the drafts or biased are special: a workgroup lists the special tokens of its range, a
// thread each forms their x (the loads of the logit and of the count on their way at
// once), and each is added to the sums and written by itself, behind the rest.  With a
// copy of the row in registers and a third of the waves in its place 1663 rows of 131072
// bf16 values took 329 us for 281 now, 194 without history, biases and masks; 176 is what
// the bytes take at a copy's 5.12 TB/s.
#include "logits_internal.h"
#include "ssu_device.cuh"

#include "../../include/ssu_logits.h"

#include <float.h>

namespace ssu {

namespace {

// ---------------------------------------------------------------------------
// histories
// ---------------------------------------------------------------------------

// Tokens [first, first + n) of entry b; false (and said so) where they are not what they have to be.
__device__ __forceinline__ bool count_range(const KHistory &h, const KCount &c, int b, int tid, int64_t &first, int &n) {
  bool ok;
  if (c.cu) {
    const int b0 = c.cu[b], b1 = c.cu[b + 1];
    ok = b0 >= 0 && b0 <= b1 && b1 <= c.rows;
    first = b0;
    n = b1 - b0;
  } else {
    first = (int64_t)b * c.T;
    n = c.num ? c.num[b] : c.T;
    ok = n >= 0 && n <= c.T;
  }
  if (!ok && tid == 0 && h.status) atomicOr(h.status, SSU_STATUS_BAD_SEQLEN);
  return ok;
}

// A workgroup per entry.  A word of `counts` whose bit was not set yet is
// emptied by the one thread that sets the bit, then all tokens are added:
// nothing but the bits has to be cleared for a new request.  A chain of a few dependent
// loads and atomics: 6.5 us for 256 entries of up to 8 tokens.
template <int NT>
__global__ __launch_bounds__(NT) void count_kernel(KHistory h, KCount c) {
  const int b = blockIdx.x, tid = threadIdx.x, slot = c.slot_idx[b];
  if (slot <= 0 || slot >= h.num_slots) return;
  int64_t first;
  int n;
  if (!count_range(h, c, b, tid, first, n)) return;
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

// A prompt's tokens, each counted once: a workgroup per entry collects their bits in
// LDS, as many words as there are, and adds them to the page without an atomic (a
// text's frequent tokens share a few words: 32 prompts of 2048 to 4096 tokens take 11 us,
// and 48 in count_kernel, which has an atomic for each token and takes the vocabularies
// of more words than there are here).
constexpr int kPromptWords = 4096;
template <int NT>
__global__ __launch_bounds__(NT) void count_prompt_kernel(KHistory h, KCount c) {
  __shared__ uint32_t mine[kPromptWords];
  const int b = blockIdx.x, tid = threadIdx.x, slot = c.slot_idx[b];
  if (slot <= 0 || slot >= h.num_slots) return;
  int64_t first;
  int n;
  if (!count_range(h, c, b, tid, first, n)) return;
  for (int w = tid; w < h.words; w += NT) mine[w] = 0;
  __syncthreads();
  const int32_t *tokens = c.tokens + first;
  bool bad = false;
  for (int i = tid; i < n; i += NT) {
    const int tok = tokens[i];
    const bool in = tok >= 0 && tok < h.vocab;
    bad |= !in;
    if (in) atomicOr(&mine[tok >> 5], 1u << (tok & 31));
  }
  if (bad && h.status) atomicOr(h.status, SSU_STATUS_BAD_TOKEN);
  __syncthreads();
  uint32_t *seen = h.seen + (int64_t)slot * h.seen_stride;
  int32_t *counts = h.counts + (int64_t)slot * h.counts_stride;
  for (int w = tid; w < h.words; w += NT) {
    const uint32_t add = mine[w], old = c.reset ? 0u : seen[w];
    if (c.reset || (add & ~old)) seen[w] = old | add;
    for (uint32_t v = add; v; v &= v - 1) {
      const int k = __builtin_ctz(v);
      int32_t *at = counts + 32 * w + k;
      *at = (old >> k) & 1u ? *at | 1 : 1;
    }
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
  // (what was unpacked of them is not worth its registers until they are wanted again)
  __device__ __forceinline__ void again() {
#pragma unroll
    for (u32x4 &v : w) asm volatile("" : "+v"(v));
  }
  __device__ __forceinline__ void load(const uint8_t *row, int i) {
    const uint8_t *at = row + (int64_t)i * logit_size(IT);
    w[0] = *reinterpret_cast<const u32x4_any *>(at);
    if constexpr (IT == kLF32) w[1] = *reinterpret_cast<const u32x4_any *>(at + 16);
  }
};

template <int OT>
__device__ __forceinline__ void store1(uint8_t *row, int i, float v) {
  if constexpr (OT == kLF32)
    reinterpret_cast<float *>(row)[i] = v;
  else
    reinterpret_cast<uint16_t *>(row)[i] = (uint16_t)(OT == kLBF16 ? pack_bf16(v, 0.f) : pack_f16(v, 0.f));
}
__device__ __forceinline__ void store16(uint8_t *at, u32x4 v, bool past) {
  if (past)
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(at));
  else
    *reinterpret_cast<u32x4_any *>(at) = v;
}
// past: by the caches
template <int OT>
__device__ __forceinline__ void store8(uint8_t *row, int i, const float (&v)[8], bool past) {
  uint8_t *at = row + (int64_t)i * logit_size(OT);
  u32x4 a;
  if constexpr (OT == kLF32) {
    u32x4 b;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = __float_as_uint(v[k]);
      b[k] = __float_as_uint(v[4 + k]);
    }
    store16(at + 16, b, past);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = OT == kLBF16 ? pack_bf16(v[2 * k], v[2 * k + 1]) : pack_f16(v[2 * k], v[2 * k + 1]);
  }
  store16(at, a, past);
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
  const uint32_t *mask;   // NULL: all
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
  r.mask = l.mask ? l.mask + r.row * l.mask_stride : nullptr;
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

// The special tokens of the values [i0, i0 + 32 * words) of a row, CAP of them at a time.
template <int NT, int WORDS, int CAP>
struct Special {
  uint32_t bits[WORDS];     // special
  uint32_t out[WORDS];      // special, or left out by the mask
  uint32_t rank[WORDS / 2]; // special ones before every other word
  uint32_t info[CAP];       // 256 (its last bias + 1) + its drafts, later x
  uint32_t token[CAP];      // in the range
  int sums[NT / 64];

  __device__ __forceinline__ int at(int o) const {  // rank of the range's value o
    const int w = o >> 5;
    return (int)rank[w >> 1] + ((w & 1) ? __builtin_popcount(bits[w - 1]) : 0) + __builtin_popcount(bits[w] & ((1u << (o & 31)) - 1u));
  }
  // The words of a thread, an even one first and an even number of them but for the last.
  static __device__ __forceinline__ void share(int words, int tid, int &w0, int &w1) {
    const int each = (words + 2 * NT - 1) / (2 * NT) * 2;
    w0 = min(tid * each, words);
    w1 = min(w0 + each, words);
  }
  __device__ __forceinline__ float x(int j) const { return __uint_as_float(info[j]); }
  // which of values o .. o + 7 of the range are not taken as they are
  __device__ __forceinline__ uint32_t out8(int o) const { return reinterpret_cast<const uint8_t *>(out)[o >> 3]; }

  // By the whole workgroup: the bitmaps; the number of special tokens.
  __device__ __forceinline__ int mark(const Row &r, int i0, int words, int vocab, int tid) {
    const int end = min(i0 + 32 * words, vocab);
    const bool some = r.seen || r.nd > 0 || r.nb > 0 || (end == vocab && (vocab & 7));
    for (int w = tid; w < words; w += NT) {
      const int left = vocab - i0 - 32 * w;  // (> 0: the words are the vocabulary's)
      const uint32_t real = left < 32 ? (1u << left) - 1u : ~0u;
      // (the row's last values that are no eight go with the special ones)
      bits[w] = (r.seen ? r.seen[(i0 >> 5) + w] & real : 0u) | (left < 32 ? real & ~((1u << (left & 24)) - 1u) : 0u);
      out[w] = r.mask ? ~r.mask[(i0 >> 5) + w] : 0u;
    }
    __syncthreads();
    if (!some) return 0;
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
    const int lane = tid & 63;
    int w0, w1, mine = 0;
    share(words, tid, w0, w1);
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
    for (int w = w0; w < w1; ++w) {
      if (!(w & 1)) rank[w >> 1] = (uint32_t)before;
      before += __builtin_popcount(bits[w]);
    }
    return total;
  }

  // By the whole workgroup: special tokens first .. first + n - 1 with their x (-inf where the mask takes them or it is
  // NaN), and into `out`.  (n <= CAP; all have read what was there.)
  template <int IT>
  __device__ __forceinline__ void form(const Row &r, int i0, int words, int vocab, int first, int n, int tid) {
    const int end = min(i0 + 32 * words, vocab);
    int w0, w1, j = 0;
    share(words, tid, w0, w1);
    if (w0 < w1) j = (int)rank[w0 >> 1] - first;
    for (int w = w0; w < w1; ++w) {
      for (uint32_t v = bits[w]; v; v &= v - 1, ++j)
        if (j >= 0 && j < n) {
          token[j] = 32 * w + __builtin_ctz(v);
          info[j] = 0;
        }
    }
    __syncthreads();
    if (r.nb > 0) {
      for (int j = tid; j < r.nb; j += NT) {
        const int k = r.bias_tok[j];
        if (k < i0 || k >= end) continue;
        const int p = at(k - i0) - first;
        if (p >= 0 && p < n) atomicMax(&info[p], (uint32_t)(j + 1) << 8);
      }
      __syncthreads();
    }
    if (r.nd > 0) {
      for (int j = tid; j < r.nd; j += NT) {
        const int k = r.drafts[j];
        if (k < i0 || k >= end) continue;
        const int p = at(k - i0) - first;
        if (p >= 0 && p < n) atomicAdd(&info[p], 1u);
      }
      __syncthreads();
    }
    for (int j = tid; j < n; j += NT) {
      const int o = token[j], i = i0 + o;
      const uint32_t f = info[j];
      const float v = logit_at<IT>(r.in, i);
      int m = (int)(f & 255u);
      bool was = m > 0;
      if (r.seen) {
        const int c = r.counts[i] >> 1;  // (loaded with the logit)
        if ((r.seen[i >> 5] >> (i & 31)) & 1u) {
          was = true;
          m += c;
        }
      }
      const bool taken = !r.mask || ((r.mask[i >> 5] >> (i & 31)) & 1u);
      const float y = special_x(r, v, f >> 8, f >> 8 ? r.bias_val[(f >> 8) - 1] : 0.f, was, m);
      info[j] = __float_as_uint(taken && y == y ? y : -INFINITY);
      atomicOr(&out[o >> 5], 1u << (o & 31));
    }
    __syncthreads();
  }
};

// Eight values of a row, NaN where the byte has a bit: it counts for nothing below.
template <int IT>
__device__ __forceinline__ void values8(const Eight<IT> &e, uint32_t out, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(__float_as_uint(e.value(k)) | (uint32_t)((int32_t)(out << (31 - k)) >> 31));
}

// The largest x and the sum of exp((x - m) / temperature), of the finite m next to it.
struct Stat {
  float m, s;
};
constexpr Stat kNoStat = {-INFINITY, 0.f};
// 2 log2(e) / temperature, finite and positive: half of x - m times it is 0 at x = m and -inf at x = -inf
__device__ __forceinline__ float slope(float temperature) {
  return fminf(fmaxf(2.8853900817779268f / temperature, FLT_TRUE_MIN), FLT_MAX);
}
// half of x - m (all of it may be no finite number, and matters where the temperature is as large)
__device__ __forceinline__ float half_of(float x, float m) { return fmaf(x, 0.5f, -0.5f * m); }
__device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -FLT_MAX), FLT_MAX); }
// exp2 between 0 and 1, 0 of NaN: of x = +inf and the largest finite m 1.  (The bounds are the instruction's own.)
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_fmed3f(__builtin_amdgcn_exp2f(d), 0.f, 1.f); }
__device__ __forceinline__ Stat join(Stat a, Stat b, float k) {
  const float m = fmaxf(a.m, b.m), M = finite(m);
  return Stat{m, a.s * exp_of(half_of(a.m, M) * k) + b.s * exp_of(half_of(b.m, M) * k)};
}
template <int N>
__device__ __forceinline__ void add_values(Stat &o, const float *v, float k) {
  float m = o.m;
#pragma unroll
  for (int e = 0; e < N; ++e) m = fmaxf(m, v[e]);
  const float M = finite(m);
  float s = o.s * exp_of(half_of(o.m, M) * k);
#pragma unroll
  for (int e = 0; e < N; ++e) s += exp_of(half_of(v[e], M) * k);
  o.m = m;
  o.s = s;
}
__device__ __forceinline__ Stat wave_join(Stat s, float k) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s = join(s, Stat{__shfl_xor(s.m, d), __shfl_xor(s.s, d)}, k);
  return s;
}
// In every thread.
template <int NT>
__device__ __forceinline__ Stat block_join(Stat s, Stat *lds, int tid, float k) {
  s = wave_join(s, k);
  __syncthreads();
  if ((tid & 63) == 0) lds[tid >> 6] = s;
  __syncthreads();
  Stat o = lds[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) o = join(o, lds[w], k);
  return o;
}

// A greedy row, temperature <= 0 or NaN: the largest x (at most the largest finite) above -inf and its lowest place.
__device__ __forceinline__ bool is_greedy(float temperature) { return !(temperature > 0.f); }
struct Best {
  float m;
  int i;
};
constexpr Best kNoBest = {-INFINITY, 0x7fffffff};
__device__ __forceinline__ Best better(Best a, Best b) { return b.m > a.m || (b.m == a.m && b.i < a.i) ? b : a; }
__device__ __forceinline__ void add_best(Best &o, float x, int i) {
  if (x > -INFINITY) o = better(o, Best{fminf(x, FLT_MAX), i});
}
template <int NT>
__device__ __forceinline__ Best block_best(Best s, Best *lds, int tid) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s = better(s, Best{__shfl_xor(s.m, d), __shfl_xor(s.i, d)});
  __syncthreads();
  if ((tid & 63) == 0) lds[tid >> 6] = s;
  __syncthreads();
  Best o = lds[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) o = better(o, lds[w]);
  return o;
}

// The probabilities of a row: exp((x - m) / temperature) / sum.
struct Probs {
  float M, k, inv;
  __device__ __forceinline__ Probs(Stat s, float slope) : M(finite(s.m)), k(slope), inv(s.m > -INFINITY ? 1.f / s.s : 0.f) {}
  __device__ __forceinline__ float operator()(float x) const { return exp_of(half_of(x, M) * k) * inv; }
};

// Says so where an entry's biased tokens are none.
__device__ __forceinline__ void bad_biases(const Row &r, const KLogits &l, int tid, int nthreads) {
  bool bad = false;
  for (int j = tid; j < r.nb; j += nthreads) bad |= r.bias_tok[j] < 0 || r.bias_tok[j] >= l.vocab;
  if (bad) atomicOr(l.status, SSU_STATUS_BAD_BIAS);
}

// All stores of the workgroup have arrived, so that others to the same places come behind them.
__device__ __forceinline__ void stores_done() {
  __threadfence_block();
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

constexpr int kPieceThreads = 256;
enum Mode { kStats, kProbs, kPlain };

// A piece of a row, 8 values a thread.  kStats: its statistics into the workspace; kProbs: its probabilities from those of
// all pieces; kPlain: x / temperature.
template <int IT, int OT, Mode MODE>
__global__ __launch_bounds__(kPieceThreads) void logits_piece_kernel(KHistory h, KLogits l, int pieces) {
  constexpr int NT = kPieceThreads;
  typedef Special<NT, kLogitsPiece / 32, kLogitsPiece> Sp;
  static_assert(kLogitsPiece == NT * 8, "8 values a thread");
  __shared__ Sp sp;
  __shared__ Stat red[NT / 64];
  const int tid = threadIdx.x, piece = blockIdx.x, b = blockIdx.y / l.T, t = blockIdx.y - b * l.T;
  Row r;
  if (!find_row(h, l, b, t, piece == 0 && tid == 0 && MODE != kProbs, r)) return;
  const int i0 = piece * kLogitsPiece, words = (min(kLogitsPiece, l.vocab - i0) + 31) / 32, i = i0 + tid * 8;
  const bool full = i + 8 <= l.vocab, greedy = is_greedy(r.temperature);
  Eight<IT> e;
  if (full) e.load(r.in, i);
  const float k = slope(r.temperature);
  uint8_t *out = l.out + r.row * l.out_stride;
  float2 *ws = l.ws + (int64_t)blockIdx.y * pieces;
  Stat s = kNoStat;
  Best best = kNoBest;
  if constexpr (MODE == kProbs) {
    for (int j = tid; j < pieces; j += NT) {
      const float2 w = ws[j];
      if (greedy)
        best = better(best, Best{w.x, (int)__float_as_uint(w.y)});
      else
        s = join(s, Stat{w.x, w.y}, k);
    }
  }
  const int total = sp.mark(r, i0, words, l.vocab, tid);
  if (total > 0) sp.template form<IT>(r, i0, words, l.vocab, 0, total, tid);
  float v[8];
  if (full) values8<IT>(e, sp.out8(tid * 8), v);
  if (MODE != kPlain && greedy) {
    if constexpr (MODE == kStats) {
      if (full) {
#pragma unroll
        for (int x = 0; x < 8; ++x) add_best(best, v[x], i + x);
      }
      for (int j = tid; j < total; j += NT) add_best(best, sp.x(j), i0 + (int)sp.token[j]);
    }
    best = block_best<NT>(best, reinterpret_cast<Best *>(red), tid);
    if (MODE == kStats && tid == 0) ws[piece] = float2{best.m, __uint_as_float((uint32_t)best.i)};
    if constexpr (MODE == kProbs) {
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = i + x == best.i ? 1.f : 0.f;
      if (full) store8<OT>(out, i, v, l.past);
      if (!full) {
        for (int x = 0; i + x < l.vocab; ++x) store1<OT>(out, i + x, i + x == best.i ? 1.f : 0.f);
      }
    }
    s.m = best.m;
  } else if constexpr (MODE == kStats) {
    if (full) add_values<8>(s, v, k);
    for (int j = tid; j < total; j += NT) {
      const float x = sp.x(j);
      add_values<1>(s, &x, k);
    }
    s = block_join<NT>(s, red, tid, k);
    if (tid == 0) ws[piece] = float2{s.m, s.s};
  } else {
    if constexpr (MODE == kProbs) s = block_join<NT>(s, red, tid, k);
    const Probs p(s, k);
    auto result = [&](float x) {
      if constexpr (MODE == kProbs) return p(x);
      const float y = greedy ? x : x / r.temperature;
      return x > -INFINITY ? y : -INFINITY;  // (NaN, and -inf also where the temperature is infinite)
    };
    if (full) {
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = result(v[x]);
      store8<OT>(out, i, v, l.past);
    }
    if (total > 0) stores_done();
    for (int j = tid; j < total; j += NT) store1<OT>(out, i0 + (int)sp.token[j], result(sp.x(j)));
  }
  if (MODE == kProbs && piece == 0 && tid == 0 && l.status && !(s.m > -INFINITY)) atomicOr(l.status, SSU_STATUS_EMPTY_ROW);
  if (MODE != kProbs && piece == 0 && l.status && r.nb > 0 && t == 0) bad_biases(r, l, tid, NT);
}

// A whole row by one workgroup, two of 16 waves a CU: enough loads on their way while the other one lists its special
// tokens.  The first HOLD groups of 8 values a thread are loaded once the special ones are marked and stay in registers, the
// others are read AHEAD at a time, and for the second time from the caches.  (512 threads and 16 groups held took 318 us for
// 289 with 1663 rows of 131072, one group at a time 304.)  ALONE: no more rows than CUs, and twice the registers for loads on
// their way (256 rows of 100003 fp32 values that no cache holds 75 -> 63 us; 16-bit ones the same as without).
// Two workgroups a CU leave room for the bitmaps and lists of 131072 values (72 KiB each).  Longer rows go by pieces, however
// many they are, which reads them once more and lists their special tokens twice (bf16, history, masks, biases: 256 rows of
// 131072 values 50 us, of 151936 135).
constexpr int kRowThreads = 1024, kRowMax = 131072, kAlone = 256;

template <int IT, int OT, bool ALONE>
__global__ __launch_bounds__(kRowThreads, ALONE ? 4 : 8) void logits_row_kernel(KHistory h, KLogits l) {
  constexpr int NT = kRowThreads, GROUP = NT * 8, HOLD = ALONE ? 8 : IT == kLF32 ? 2 : 4, AHEAD = HOLD / 2, CAP = 4096;
  typedef Special<NT, kRowMax / 32, CAP> Sp;
  __shared__ Sp sp;
  __shared__ Stat red[NT / 64];
  const int tid = threadIdx.x, b = blockIdx.x / l.T, t = blockIdx.x - b * l.T;
  Row r;
  if (!find_row(h, l, b, t, tid == 0, r)) return;
  const int vocab = l.vocab, words = (vocab + 31) / 32, whole = vocab & ~7;
  const float k = slope(r.temperature);
  uint8_t *out = l.out + r.row * l.out_stride;
  const int total = sp.mark(r, 0, words, vocab, tid);
  // the special tokens, as many at a time as LDS has room for
  auto special = [&](auto use) {
    for (int first = 0; first < total; first += CAP) {
      const int n = min(CAP, total - first);
      sp.template form<IT>(r, 0, words, vocab, first, n, tid);
      for (int j = tid; j < n; j += NT) use(sp.x(j), (int)sp.token[j]);
      if (total > CAP) __syncthreads();
    }
  };
  if (l.status && r.nb > 0 && t == 0) bad_biases(r, l, tid, NT);
  if (is_greedy(r.temperature)) {
    Best best = kNoBest;
    special([&](float x, int i) { add_best(best, x, i); });
    for (int i = tid * 8; i < whole; i += GROUP) {
      Eight<IT> w;
      w.load(r.in, i);
      float v[8];
      values8<IT>(w, sp.out8(i), v);
#pragma unroll
      for (int x = 0; x < 8; ++x) add_best(best, v[x], i + x);
    }
    best = block_best<NT>(best, reinterpret_cast<Best *>(red), tid);
    for (int i = tid * 8; i < whole; i += GROUP) {
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = i + x == best.i ? 1.f : 0.f;
      store8<OT>(out, i, v, l.past);
    }
    if (tid < vocab - whole) store1<OT>(out, whole + tid, whole + tid == best.i ? 1.f : 0.f);
    if (tid == 0 && l.status && !(best.m > -INFINITY)) atomicOr(l.status, SSU_STATUS_EMPTY_ROW);
    return;
  }
  Eight<IT> e[HOLD];
#pragma unroll
  for (int g = 0; g < HOLD; ++g) {
    const int i = g * GROUP + tid * 8;
    if (i < whole) e[g].load(r.in, i);
  }
  Stat s = kNoStat;
  special([&](float x, int) { add_values<1>(s, &x, k); });
  auto groups = [&](auto use) {
#pragma unroll
    for (int g = 0; g < HOLD; ++g) {
      const int i = g * GROUP + tid * 8;
      if (i < whole) use(e[g], i);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int i0 = HOLD * GROUP + tid * 8; i0 < whole; i0 += AHEAD * GROUP) {
      Eight<IT> w[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a)
        if (i0 + a * GROUP < whole) w[a].load(r.in, i0 + a * GROUP);
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        if (i0 + a * GROUP < whole) use(w[a], i0 + a * GROUP);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  groups([&](const Eight<IT> &w, int i) {
    float v[8];
    values8<IT>(w, sp.out8(i), v);
    add_values<8>(s, v, k);
  });
  s = block_join<NT>(s, red, tid, k);
  const Probs p(s, k);
#pragma unroll
  for (int g = 0; g < HOLD; ++g) e[g].again();
  // Where the list is not all of them, the special ones are formed again and written first (their logits may lie where the
  // probabilities go), and the others around them.
  if (total > CAP) {
    special([&](float x, int i) { store1<OT>(out, i, p(x)); });
    groups([&](const Eight<IT> &w, int i) {
      float v[8];
      values8<IT>(w, sp.out8(i), v);
      const uint32_t around = (sp.bits[i >> 5] >> (i & 31)) & 255u;
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (!((around >> x) & 1u)) store1<OT>(out, i + x, p(v[x]));
    });
  } else {
    groups([&](const Eight<IT> &w, int i) {
      float v[8];
      values8<IT>(w, sp.out8(i), v);
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = p(v[x]);
      store8<OT>(out, i, v, l.past);
    });
    if (total > 0) {
      stores_done();
      for (int j = tid; j < total; j += NT) store1<OT>(out, (int)sp.token[j], p(sp.x(j)));
    }
  }
  if (tid == 0 && l.status && !(s.m > -INFINITY)) atomicOr(l.status, SSU_STATUS_EMPTY_ROW);
}

template <int IT, int OT>
hipError_t logits_t(const KHistory &h, const KLogits &l, bool softmax, hipStream_t st) {
  const int pieces = (l.vocab + kLogitsPiece - 1) / kLogitsPiece, rows = l.batch * l.T;
  const dim3 grid((unsigned)pieces, (unsigned)rows), block(kPieceThreads);
  if (!softmax) {
    logits_piece_kernel<IT, OT, kPlain><<<grid, block, 0, st>>>(h, l, pieces);
    return hipGetLastError();
  }
  // One launch against two and a read more, with 131072 bf16 values a row (f32 out) 64 rows 38.5 : 38.6 us, 32 rows 34 : 23,
  // 256 rows 54 : 116; with 32000 32 rows 15.7 : 15.8, 1 row 14.3 : 13.0; with 8000 1 row 11.7 : 13.4, 64 rows 13.0 : 15.8.
  if (l.vocab <= kRowMax && (rows >= pieces || l.vocab <= 16384)) {
    if (rows <= kAlone)
      logits_row_kernel<IT, OT, true><<<dim3((unsigned)rows), dim3(kRowThreads), 0, st>>>(h, l);
    else
      logits_row_kernel<IT, OT, false><<<dim3((unsigned)rows), dim3(kRowThreads), 0, st>>>(h, l);
    return hipGetLastError();
  }
  logits_piece_kernel<IT, kLF32, kStats><<<grid, block, 0, st>>>(h, l, pieces);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  logits_piece_kernel<IT, OT, kProbs><<<grid, block, 0, st>>>(h, l, pieces);
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
  if (c.prompt && h.words <= kPromptWords)
    count_prompt_kernel<1024><<<dim3((unsigned)c.batch), dim3(1024), 0, st>>>(h, c);
  else if (!c.reset && !c.cu && c.T <= 64)
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
