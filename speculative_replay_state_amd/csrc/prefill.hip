// The selective state update over whole sequences, in chunks of 64 tokens.
//
// With G_t the running sum of A dt' within a chunk (fp64, in units of ln 2),
//   y_t = e^(G_t) C_t.S + sum_(s <= t) W_ts x_s,
//   W_ts = e^(G_t - G_s) dt'_s (C_t.B_s), + D on the diagonal,
//   S' = e^(G_w) S + sum_s (e^(G_w - G_s) dt'_s x_s) B_s^T.
// Everything but the exponentials is matrix products: a chunk and a head cost 192 products of
// 16 x 16 x 32 for the readout, 192 for the update, 72 for the tokens of the chunk and 64 for
// C.B, which the heads of a workgroup share.  Their operands that are not bf16 have to be split
// into three bf16 parts on the way, and that and the weights cost the vector units more again:
// 8 prompts of 2048 to 4096 tokens of 128 heads take 475 us, 186 are their bytes, 157 the
// products alone at 2.5 PFLOP/s; matrix units are busy for 35 % of it, vector units for 38, and
// the two waves of a SIMD issue for 35 % of theirs, wait for a busy unit or a result for 43, and
// for loads and barriers for 21.
// Two waves a head have 32 of its 64 columns each (or four have 16), the state in registers
// as matrix results [n][p], which are the next product's operand as they lie.  B, C and x of a
// chunk lie in LDS, the next chunk's on their way in registers.
//
// Long sequences are cut into segments: prefill_kernel<.., true> forms what each
// segment but the last adds to the state and its decay, segment_kernel the state that
// each starts from, then all segments run at once (16384 tokens of 64 heads, gated: 65, 13 and
// 188 of 263 us).
#include <stddef.h>

#include <algorithm>

#include "delta_device.cuh"
#include "prefill_internal.h"

namespace ssu {

namespace {

constexpr int kT = kPChunk / 16;              // token tiles of a chunk
constexpr int kTiles = kT * (kT + 1) / 2;     // C.B tiles on and below the diagonal
constexpr int kHeadValues = kHeadDim * kDState;
constexpr int head_waves(int CT) { return kT / CT; }  // of a head, 16 CT columns each: they form the gates of as many chunks at once

// bf16 parts of an operand that is not bf16: 24 bits, whatever the outputs' type (with two, off by 2^-18, bf16 outputs round
// the other way often enough to end 1.0e-4 of the norm from the rounded exact ones, for 2.8e-5 with three).
constexpr int kParts = 3;

// [b0, b1) of sequence s; false where cu_seqlens is not what it has to be.
__device__ __forceinline__ bool seq_rows(const KPrefill &p, int s, int &b0, int &b1) {
  b0 = p.cu[s];
  b1 = p.cu[s + 1];
  return b0 >= 0 && b0 <= b1 && b1 <= p.rows;
}
// Segments of a sequence of `len` tokens: up to two segments' tokens stay together.
__device__ __forceinline__ int segments_of(const KPrefill &p, int64_t len) {
  return len <= 2 * (int64_t)p.seg ? 1 : (int)((len + p.seg - 1) / p.seg);
}

struct Segment {
  int seq, i, n;  // the i-th of n segments of the sequence
  int b0, b1;     // the sequence's rows
};

__device__ __forceinline__ int slot_base(const KPrefill &p, int s) { return max(p.cu[s], 0) / p.seg + s; }

// By a whole wave: what lies in a slot; false where nothing does.  Up to 64 sequences: their segments
// one after the other, the longest sequences first.  More: as they come, from slot_base on (a sequence
// has at most len / seg + 1 segments, so the slots of two sequences differ).
__device__ __forceinline__ bool find_segment(const KPrefill &p, int slot, int lane, Segment &o) {
  if (p.n <= 64) {
    const int s = min(lane, p.n - 1);
    const bool ok = seq_rows(p, s, o.b0, o.b1) && lane < p.n;
    const int len = ok ? o.b1 - o.b0 : -1, mine = ok ? segments_of(p, len) : 0;
    int first = 0;
    for (int t = 0; t < p.n; ++t) {
      const int other = __builtin_amdgcn_readlane(len, t);
      first += other > len || (other == len && t < lane) ? __builtin_amdgcn_readlane(mine, t) : 0;
    }
    const uint64_t in = __ballot(first <= slot && slot < first + mine);
    if (in == 0) return false;
    o.seq = __builtin_ctzll(in);
    o.i = slot - __builtin_amdgcn_readlane(first, o.seq);
    o.n = __builtin_amdgcn_readlane(mine, o.seq);
    return seq_rows(p, o.seq, o.b0, o.b1);
  }
  int lo = 0, hi = p.n;  // the last sequence whose first slot is at most `slot`
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int64_t s = lo + (int64_t)lane * step;
    const uint64_t in = __ballot(s < hi && slot_base(p, (int)min(s, (int64_t)p.n - 1)) <= slot);
    if (in == 0) return false;
    lo += (63 - __builtin_clzll(in)) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  o.seq = lo;
  if (!seq_rows(p, lo, o.b0, o.b1)) return false;
  o.i = slot - slot_base(p, lo);
  o.n = segments_of(p, o.b1 - o.b0);
  return o.i < o.n;
}
// The first slot of sequence s (by a whole wave, where it has one).
__device__ __forceinline__ int first_slot(const KPrefill &p, int s, int lane) {
  if (p.n > 64) return slot_base(p, s);
  int b0, b1;
  const bool ok = seq_rows(p, min(lane, p.n - 1), b0, b1) && lane < p.n;
  const int len = ok ? b1 - b0 : -1, mine = ok ? segments_of(p, len) : 0, of = __builtin_amdgcn_readlane(len, s);
  int first = len > of || (len == of && lane < s) ? mine : 0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) first += __shfl_xor(first, d);
  return first;
}

// What a head's tokens of a chunk contribute, in LDS.  G_t - G_s of tokens in
// one tile of 16 is taken as hi_t - hi_s + (lo_t - lo_s), which keeps fp32 accuracy of the
// difference; of tokens in two, by way of the border before t's tile.
struct Gates {
  float hi[kPChunk], lo[kPChunk], dt[kPChunk];  // G in two parts; dt'
  float w[kPChunk], e[kPChunk];                 // e^(G_w - G) dt', e^G
  float row[kPChunk];                           // e^(G - G before the token's tile)
  float col[kT - 1][kPChunk];                   // e^(G before tile ti - G) dt', for the tokens before tile ti = 1, 2, 3
  float last[4];                                // e^(G_w)
};

// Rows in LDS.  B and C: 32 bytes apart from a multiple of all banks (8 rows of 16 bytes do not meet in one); x, whose
// rows are half as long, with its pieces of 16 bytes moved by the row.
constexpr int kBcRow = kDState + 16;
__device__ __forceinline__ int bc_piece(int t, int piece) { return t * kBcRow + 8 * piece; }
__device__ __forceinline__ int x_piece(int t, int piece) { return t * kHeadDim + ((piece ^ (t & 6)) << 3); }

template <int HPW, bool STATE>
struct PBuf {
  __align__(16) uint16_t B[kPChunk * kBcRow], C[STATE ? 8 : kPChunk * kBcRow], x[HPW][kPChunk * kHeadDim];
};

// The pairs of a chunk's tiles of 16 tokens ti with tiles of 32 ks that hold tokens up to them.
constexpr int kPairs = 6;
constexpr int pair_at(int ti, int ks) { return (ti < 2 ? ti : 2 * ti - 2) + ks; }
// A head's W of a chunk as the parts of operands: they take the place of C and x, which nobody reads any more by then.
constexpr size_t kHeadWeights = kPairs * kParts * 64 * sizeof(bf16x8);

// v of lane l
__device__ __forceinline__ double lane_d(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, l), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sums of the lanes up to and with this one.
__device__ __forceinline__ double scan64(double v, int lane) {
  v += row_shr_d<1>(v);
  v += row_shr_d<2>(v);
  v += row_shr_d<4>(v);
  v += row_shr_d<8>(v);
  const double r0 = lane_d(v, 15), r1 = lane_d(v, 31), r2 = lane_d(v, 47);
  double add = lane >= 16 ? r0 : 0.0;
  if (lane >= 32) add += r1;
  if (lane >= 48) add += r2;
  return v + add;
}

// log(1 + e^v) with no branch: max(v, 0) + log(1 + u), u = e^-|v| in (0, 1], the logarithm by the series of its
// inverse hyperbolic tangent, 2 (s + s^3 / 3 + s^5 / 5 + ...) at s = u / (2 + u) <= 1/3 (a part in 2^27 behind
// s^17), within a few units of the last place.
__device__ __forceinline__ float softplus_series(float v) {
  const float a = fminf(fabsf(v), 126.f), p = a * -1.44269502f;
  const float rest = fmaf(a, -1.44269502f, -p) + a * -1.92596303e-8f;  // what p leaves of a log2(e)
  const float u0 = __builtin_amdgcn_exp2f(p), u = fmaf(u0, rest * 0.69314718f, u0);
  const float den = 2.f + u, r0 = __builtin_amdgcn_rcpf(den), r = fmaf(fmaf(-den, r0, 1.f), r0, r0);
  const float s = u * r, q = s * s;
  float t = 1.f / 17.f;
  t = fmaf(t, q, 1.f / 15.f);
  t = fmaf(t, q, 1.f / 13.f);
  t = fmaf(t, q, 1.f / 11.f);
  t = fmaf(t, q, 1.f / 9.f);
  t = fmaf(t, q, 1.f / 7.f);
  t = fmaf(t, q, 1.f / 5.f);
  t = fmaf(t, q, 1.f / 3.f);
  const float s2 = s + s, l = fmaf(s2 * q, t, s2);
  return v == v ? (v > 0.f ? v : 0.f) + l : v;
}

// By a wave: the gates of a chunk (lane = token, `there` of them with one); the log2 of its whole decay.
template <bool STATE>
__device__ __forceinline__ double write_gates(Gates &g, float dt, float bias, float A, int softplus, int there, int lane) {
  const float v = dt + bias;
  const float d = lane < there ? (softplus ? softplus_series(v) : v) : 0.f;
  double a = (double)A * d;
  a = lane < there ? (a < -0x1p20 ? -0x1p20 : a) : 0.0;  // (NaN stays)
  const double G = scan64(a * kLog2e, lane), Gw = lane_d(G, 63);
  if constexpr (!STATE) {
    const float hi = (float)G;
    g.hi[lane] = hi;
    g.lo[lane] = (float)(G - (double)hi);
    g.dt[lane] = d;
    g.e[lane] = exp2_d(G);
    double border = 0.0;
#pragma unroll
    for (int ti = 1; ti < kT; ++ti) {
      const double b = lane_d(G, 16 * ti - 1);
      if (lane >= 16 * ti) border = b;
      if (lane < 16 * ti) g.col[ti - 1][lane] = exp2_d(b - G) * d;
    }
    g.row[lane] = exp2_d(G - border);
  }
  g.w[lane] = exp2_d(Gw - G) * d;
  if (lane == 0) g.last[0] = exp2_d(Gw);
  return Gw;
}

// Rows t0 .. t0 + 15 of B or C along n0 .. n0 + 31
__device__ __forceinline__ bf16x8 row_frag(const uint16_t *rows, int t0, int n0, int lane) {
  return __builtin_bit_cast(bf16x8, ld16(rows + bc_piece(t0 + (lane & 15), n0 / 8 + (lane >> 4))));
}
// The same transposed, tokens 32 ks .. along the depth: row m = 4 j + r of the tile is n = n0 + 8 j + 4 a + r
__device__ __forceinline__ bf16x8 b_tile(const uint16_t *B, int ks, int n0, int a, int lane) {
  const int m = lane & 15, t = 32 * ks + 4 * (lane >> 4) + (m >> 2), piece = n0 / 8 + (m & 3);
  struct { s16x4 lo, hi; } r = {lds_tr4(B + bc_piece(t, piece) + 4 * a), lds_tr4(B + bc_piece(t + 16, piece) + 4 * a)};
  return __builtin_bit_cast(bf16x8, r);
}
// Columns p .. p + 15 of x, tokens 32 ks .. along the depth
__device__ __forceinline__ bf16x8 x_tile(const uint16_t *x, int ks, int p, int lane) {
  const int m = lane & 15, t = 32 * ks + 4 * (lane >> 4) + (m >> 2), piece = p / 8 + (m >> 1 & 1), in = 4 * (m & 1);
  struct { s16x4 lo, hi; } r = {lds_tr4(x + x_piece(t, piece) + in), lds_tr4(x + x_piece(t + 16, piece) + in)};
  return __builtin_bit_cast(bf16x8, r);
}

// z sigmoid(z) times v: e^-z as 2 to an exact product of z (8 bits) and 15 bits of log2(e), times what those leave.
__device__ __forceinline__ float gated(float v, float z) {
  const float hi = -z * 0x1.7154p+0f, lo = z * -0x1.d94aep-18f;  // log2(e) = 1.44268799 + 7.0526e-6
  const float e = __builtin_amdgcn_exp2f(hi);
  return v * z * __builtin_amdgcn_rcpf(1.f + fmaf(e, lo * 0.69314718f, e));
}

// A chunk's rows on their way from memory to LDS through the registers of NT
// threads; rows behind the segment's last repeat it (their dt' is 0), heads
// behind the group's last repeat that.  Every load is unconditional.
template <int HPW, int CT, bool STATE>
struct PStage {
  static constexpr int NT = HPW * head_waves(CT) * 64;
  static constexpr int RB = NT / (kDState / 8), RX = NT / (HPW * kHeadDim / 8);  // rows that a step of all threads covers
  static constexpr int NB = kPChunk / RB, NX = kPChunk / RX;
  u32x4 b[NB], c[STATE ? 1 : NB], x[NX];
  // uniform bases of the segment's first row, bytes between rows
  const char *Bp, *Cp, *xp;
  uint32_t bs, cs, xs;
  int heads;

  __device__ __forceinline__ void begin(const KPrefill &p, int64_t row0, int g, int h0, int n) {
    Bp = reinterpret_cast<const char *>(p.B + row0 * p.B_stride + g * kDState);
    Cp = reinterpret_cast<const char *>(p.C + row0 * p.C_stride + g * kDState);
    xp = reinterpret_cast<const char *>(p.x + row0 * p.x_stride + h0 * kHeadDim);
    bs = (uint32_t)p.B_stride * 2;
    cs = (uint32_t)p.C_stride * 2;
    xs = (uint32_t)p.x_stride * 2;
    heads = n;
  }
  // rows first .. first + 63 of the segment, those behind `last` (of the 64) as that one
  __device__ __forceinline__ void fetch(int first, int last, int tid) {
    const char *B = Bp + (int64_t)first * bs, *C = Cp + (int64_t)first * cs, *X = xp + (int64_t)first * xs;
    const uint32_t tb = tid / (kDState / 8), tx = tid / (HPW * 8), ch = tid % (HPW * 8);
    const uint32_t bch = tid % (kDState / 8) * 16, xch = min((int)ch / 8, heads - 1) * 128 + ch % 8 * 16;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      b[i] = ld16(B + (uint32_t)(min(tb * bs + i * RB * bs, last * bs) + bch));
      if constexpr (!STATE) c[i] = ld16(C + (uint32_t)(min(tb * cs + i * RB * cs, last * cs) + bch));
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) x[i] = ld16(X + (uint32_t)(min(tx * xs + i * RX * xs, last * xs) + xch));
  }
  __device__ __forceinline__ void store(PBuf<HPW, STATE> &o, int tid) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int at = i * NT + tid, t = at / (kDState / 8), ch = at % (kDState / 8);
      st16(o.B + bc_piece(t, ch), b[i]);
      if constexpr (!STATE) st16(o.C + bc_piece(t, ch), c[i]);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int at = i * NT + tid, t = at / (HPW * 8), ch = at % (HPW * 8);
      st16(o.x[ch / 8] + x_piece(t, ch % 8), x[i]);
    }
  }
};

// Lane (m, q) of a wave holds of the state column p = p0 + 16 pt + m, values n =
// 32 i + 8 q + 4 a + r in S[pt][i][a][r]; of the outputs row p0 + 16 pt + 4 q + r,
// token 16 ti + m in y[pt][ti][r].
template <int OT, int HPW, int CT, bool STATE, bool GATE>
__global__ __launch_bounds__(HPW * head_waves(CT) * 64, HPW * head_waves(CT) / 2) void prefill_kernel(KPrefill p, int htiles, int unit, int64_t ntiles) {
  constexpr int NP = kParts, WPH = head_waves(CT), NT = HPW * WPH * 64;
  typedef PBuf<HPW, STATE> Buf;
  constexpr size_t kWeightsAt = offsetof(Buf, C), kWeightsEnd = STATE ? 0 : kWeightsAt + HPW * kHeadWeights;
  __shared__ __align__(16) uint8_t buf[sizeof(Buf) > kWeightsEnd ? sizeof(Buf) : kWeightsEnd];
  Buf &in = *reinterpret_cast<Buf *>(buf);
  __shared__ __align__(16) Gates gates[HPW][WPH];
  __shared__ f32x4 cb[STATE ? 1 : kTiles][64];
  static_assert(2 * (sizeof(buf) + sizeof(gates) + sizeof(cb)) <= 160 * 1024, "two workgroups a CU");
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), hh = wave / WPH, wh = wave % WPH, p0 = wh * 16 * CT;
  if (!STATE) {
    for (int64_t s = (int64_t)blockIdx.x * NT + tid; s < p.n; s += (int64_t)gridDim.x * NT) {
      int b0, b1;
      if (!seq_rows(p, (int)s, b0, b1) && p.status) atomicOr(p.status, SSU_STATUS_BAD_SEQLEN);
    }
  }
  // Units of workgroups, heads of a group on the same rows, share an XCD; the units go to the XCDs in turn.  Of an
  // XCD's 32 CUs, with room for two workgroups each, the ones that got the longest get the shortest beside them.
  int j = blockIdx.x >> 3;
  const int last_j = min((int)(gridDim.x >> 3), 64) - 1;
  if (j >= 32 && j <= last_j) j = 32 + last_j - j;
  const int64_t tile = ((int64_t)(j / unit) * 8 + (blockIdx.x & 7)) * unit + j % unit;
  if (tile >= ntiles) return;
  const int per_group = htiles / p.G;
  const int ht = (int)(tile % htiles), slot = (int)(tile / htiles);
  const int g = ht / per_group, hfirst = g * p.hpg + ht % per_group * HPW, heads = min(HPW, (g + 1) * p.hpg - hfirst);
  Segment sg;
  if (!find_segment(p, slot, lane, sg)) return;
  sg.b0 = __builtin_amdgcn_readfirstlane(sg.b0);
  sg.b1 = __builtin_amdgcn_readfirstlane(sg.b1);
  sg.seq = __builtin_amdgcn_readfirstlane(sg.seq);
  sg.i = __builtin_amdgcn_readfirstlane(sg.i);
  sg.n = __builtin_amdgcn_readfirstlane(sg.n);
  if (STATE && sg.i >= sg.n - 1) return;
  const int64_t row0 = sg.b0 + (int64_t)sg.i * p.seg;
  const int rows = (int)(sg.i < sg.n - 1 ? (int64_t)p.seg : sg.b1 - row0), chunks = (rows + kPChunk - 1) / kPChunk;
  const bool on = hh < heads;
  const int h = hfirst + min(hh, heads - 1);

  f32x4 S[CT][4][2];
  const int64_t own = (int64_t)h * kHeadValues + (p0 + m) * kDState + 8 * q;  // of (i, a, pt) = 0
  const float *from = STATE ? nullptr : (sg.n > 1 ? p.ws + (int64_t)slot * p.H * kHeadValues : p.h0 ? p.h0 + (int64_t)sg.seq * p.H * kHeadValues : nullptr);
#pragma unroll
  for (int pt = 0; pt < CT; ++pt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int a = 0; a < 2; ++a)
        S[pt][i][a] = from ? *reinterpret_cast<const f32x4 *>(from + own + pt * 16 * kDState + 32 * i + 4 * a) : f32x4{0.f, 0.f, 0.f, 0.f};

  if (chunks > 0) {
    const float A = p.A[h], bias = p.dt_bias[h], D = STATE ? 0.f : p.D[h];
    double total = 0.0;
    PStage<HPW, CT, STATE> st;
    auto last_of = [&](int c) { return min(kPChunk, rows - c * kPChunk) - 1; };
    // tokens of chunk c (0: there is none), and their dt
    auto there_of = [&](int c) { return max(0, min(kPChunk, rows - c * kPChunk)); };
    auto dt_of = [&](int c) { return p.dt[(row0 + min(c * kPChunk + lane, rows - 1)) * p.H + h]; };
    // of z and the outputs: a uniform base and the lane's offset
    constexpr int kOut = OT == kOutF32 ? 4 : 2;
    const uint32_t os = (uint32_t)p.H * kHeadDim * kOut;
    const uint32_t zs = (uint32_t)p.z_stride * 2;
    const char *zp = GATE ? reinterpret_cast<const char *>(p.z + row0 * p.z_stride) : nullptr;
    st.begin(p, row0, g, hfirst, heads);
    st.fetch(0, last_of(0), tid);
    float dt = dt_of(wh);
    for (int c = 0; c < chunks; ++c) {
      // The lane's addresses are formed again in every chunk: held from one to the next they would spill.
      int thread = tid;
      asm volatile("" : "+v"(thread));
      const int lane = thread & 63, m = lane & 15, q = lane >> 4;
      const int W = last_of(c) + 1, next = min(c + 1, chunks - 1);
      char *out = static_cast<char *>(p.out) + (row0 + c * kPChunk) * os;
      __syncthreads();
      st.store(in, thread);
      if (c % WPH == 0) {  // the gates of the next chunks, one by each of the head's waves
        const int c0 = c + wh;
        total += write_gates<STATE>(gates[hh][wh], dt, bias, A, p.softplus, there_of(c0), lane);
        dt = dt_of(c0 + WPH);
      }
      __syncthreads();
      const Gates &gt = gates[hh][c % WPH];
      u32x2 zw[CT][kT];
      if constexpr (GATE) {
        const char *z = zp + (int64_t)c * kPChunk * zs;
        const uint32_t zch = (h * kHeadDim + p0 + 4 * q) * 2;
#pragma unroll
        for (int ti = 0; ti < kT; ++ti)
#pragma unroll
          for (int pt = 0; pt < CT; ++pt) zw[pt][ti] = ld8(z + (uint32_t)(min(m * zs + 16 * ti * zs, (W - 1) * zs) + zch) + 32 * pt);
      }
      bf16x8 xf[CT][2];
#pragma unroll
      for (int pt = 0; pt < CT; ++pt)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) xf[pt][ks] = x_tile(in.x[hh], ks, p0 + 16 * pt, lane);
      f32x4 y[CT][kT];
      if constexpr (!STATE) {
        // The state's readout, and beside it C.B of the wave's token tile with all (those above the diagonal are not
        // used).  What a step reads from LDS is read a step ahead.
        static_assert(HPW * WPH == kT, "a token tile of B a wave");
        f32x4 v[kT];
#pragma unroll
        for (int ti = 0; ti < kT; ++ti) {
#pragma unroll
          for (int pt = 0; pt < CT; ++pt) y[pt][ti] = f32x4{0.f, 0.f, 0.f, 0.f};
          v[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        bf16x8 cf[2][kT], bf[2];
        auto read = [&](int i) {
          bf[i & 1] = row_frag(in.B, 16 * wave, 32 * i, lane);
#pragma unroll
          for (int ti = 0; ti < kT; ++ti) cf[i & 1][ti] = row_frag(in.C, 16 * ti, 32 * i, lane);
        };
        read(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < 3) read(i + 1);
          __builtin_amdgcn_sched_barrier(0);
          bf16x8 f[CT][NP];
#pragma unroll
          for (int pt = 0; pt < CT; ++pt) {
            const float s[8] = {S[pt][i][0][0], S[pt][i][0][1], S[pt][i][0][2], S[pt][i][0][3],
                                S[pt][i][1][0], S[pt][i][1][1], S[pt][i][1][2], S[pt][i][1][3]};
            split<NP>(s, f[pt]);
          }
#pragma unroll
          for (int ti = 0; ti < kT; ++ti) v[ti] = mfma_bf16(bf[i & 1], cf[i & 1][ti], v[ti]);
#pragma unroll
          for (int a = NP - 1; a >= 0; --a)
#pragma unroll
            for (int ti = 0; ti < kT; ++ti)
#pragma unroll
              for (int pt = 0; pt < CT; ++pt) y[pt][ti] = mfma_bf16(f[pt][a], cf[i & 1][ti], y[pt][ti]);
        }
#pragma unroll
        for (int ti = 0; ti < kT; ++ti)
          if (ti >= wave) cb[ti * (ti + 1) / 2 + wave][lane] = v[ti];
      }
      // S <- e^(G_w) S + B^T (w x)
      {
        st.fetch(next * kPChunk, last_of(next), thread);
        bf16x8 xw[CT][3], bt[3];
        auto read = [&](int j) { bt[j % 3] = b_tile(in.B, j >> 3, 32 * (j >> 1 & 3), j & 1, lane); };
        auto weigh = [&](int ks) {  // w x of tokens 32 ks .., in three parts
          const f32x4 w0 = *reinterpret_cast<const f32x4 *>(gt.w + 32 * ks + 4 * q);
          const f32x4 w1 = *reinterpret_cast<const f32x4 *>(gt.w + 32 * ks + 16 + 4 * q);
#pragma unroll
          for (int pt = 0; pt < CT; ++pt) {
            const u32x4 xx = __builtin_bit_cast(u32x4, xf[pt][ks]);
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = bf2f((xx[r >> 1] >> (16 * (r & 1))) & 0xFFFFu) * (r < 4 ? w0[r & 3] : w1[r & 3]);
            split<3>(v, xw[pt]);
          }
        };
        read(0);
        read(1);
        const float ew = gt.last[0];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int ks = j >> 3, i = j >> 1 & 3, a = j & 1;
          if (j < 14) read(j + 2);
          if (i + a == 0) weigh(ks);
          __builtin_amdgcn_sched_barrier(0);
          if (ks == 0) {
#pragma unroll
            for (int pt = 0; pt < CT; ++pt) S[pt][i][a] = scale4(S[pt][i][a], ew);
          }
#pragma unroll
          for (int k = 2; k >= 0; --k)
#pragma unroll
            for (int pt = 0; pt < CT; ++pt) S[pt][i][a] = mfma_bf16(bt[j % 3], xw[pt][k], S[pt][i][a]);
        }
      }
      if constexpr (!STATE) {
        // W of tokens 16 ti .. with 32 ks .., as the parts of an operand
        auto weights = [&](int ti, int ks, bf16x8 (&wf)[NP]) {
          const int t = 16 * ti + m;
          float w[8];
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const int si = 2 * ks + a, s0 = 16 * si + 4 * q;
            if (si > ti) {
#pragma unroll
              for (int r = 0; r < 4; ++r) w[4 * a + r] = 0.f;
              continue;
            }
            const f32x4 v = cb[ti * (ti + 1) / 2 + si][lane];
            if (si < ti) {
              const f32x4 col = *reinterpret_cast<const f32x4 *>(gt.col[ti - 1] + s0);
              const float row = gt.row[t];
#pragma unroll
              for (int r = 0; r < 4; ++r) w[4 * a + r] = v[r] * col[r] * row;
              continue;
            }
            const f32x4 shi = *reinterpret_cast<const f32x4 *>(gt.hi + s0), slo = *reinterpret_cast<const f32x4 *>(gt.lo + s0);
            const f32x4 sdt = *reinterpret_cast<const f32x4 *>(gt.dt + s0);
            const float hi = gt.hi[t], lo = gt.lo[t];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float d = __builtin_amdgcn_exp2f((hi - shi[r]) + (lo - slo[r])) * sdt[r] * v[r];
              w[4 * a + r] = 4 * q + r < m ? d : (4 * q + r == m ? d + D : 0.f);
            }
          }
          split<NP>(w, wf);
        };
        // A head's waves form a part of W each.
        bf16x8 *shared = reinterpret_cast<bf16x8 *>(buf + kWeightsAt + hh * kHeadWeights) + lane;
        __syncthreads();
        auto form = [&](int ti) {
#pragma unroll
          for (int ks = 0; ks <= ti / 2; ++ks) {
            bf16x8 wf[NP];
            weights(ti, ks, wf);
#pragma unroll
            for (int a = 0; a < NP; ++a) shared[(pair_at(ti, ks) * NP + a) * 64] = wf[a];
          }
        };
        if (wh == 0) form(0);
        if (wh == 1) form(1);
        if (wh == (CT == 2 ? 1 : 2)) form(2);
        if (wh == (CT == 2 ? 0 : 3)) form(3);
        __syncthreads();
        // the tokens of the chunk, and out
        const uint32_t och = (h * kHeadDim + p0 + 4 * q) * kOut;
#pragma unroll
        for (int ti = 0; ti < kT; ++ti) {
          const int t = 16 * ti + m;
          const float e = gt.e[t];
#pragma unroll
          for (int pt = 0; pt < CT; ++pt) y[pt][ti] = scale4(y[pt][ti], e);
#pragma unroll
          for (int ks = 0; ks <= ti / 2; ++ks) {
            bf16x8 wf[NP];
#pragma unroll
            for (int a = 0; a < NP; ++a) wf[a] = shared[(pair_at(ti, ks) * NP + a) * 64];
#pragma unroll
            for (int a = NP - 1; a >= 0; --a)
#pragma unroll
              for (int pt = 0; pt < CT; ++pt) y[pt][ti] = mfma_bf16(xf[pt][ks], wf[a], y[pt][ti]);
          }
          if (on && t < W) {
#pragma unroll
            for (int pt = 0; pt < CT; ++pt) {
              f32x4 v = y[pt][ti];
              if (GATE) {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = gated(v[r], bf2f((zw[pt][ti][r >> 1] >> (16 * (r & 1))) & 0xFFFFu));
              }
              char *at = out + (uint32_t)(m * os + och + 16 * ti * os) + 16 * pt * kOut;
              if constexpr (OT == kOutF32)
                *reinterpret_cast<f32x4 *>(at) = v;
              else
                st8(at, u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])});
            }
          }
        }
      }
    }
    if constexpr (STATE) {  // each wave has summed the chunks it formed
      __syncthreads();
      double *sum = reinterpret_cast<double *>(&gates[hh][0]);
      if (lane == 0) sum[wh] = total;
      __syncthreads();
      if (wh == 0 && lane == 0 && on) {
        total = sum[0];
#pragma unroll
        for (int k = 1; k < WPH; ++k) total += sum[k];
        p.decay[(int64_t)slot * p.H + h] = total;
      }
    }
  }
  float *to = STATE ? p.ws + (int64_t)slot * p.H * kHeadValues : (p.h1 && sg.i == sg.n - 1 ? p.h1 + (int64_t)sg.seq * p.H * kHeadValues : nullptr);
  if (!to || !on) return;
#pragma unroll
  for (int pt = 0; pt < CT; ++pt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int a = 0; a < 2; ++a) *reinterpret_cast<f32x4 *>(to + own + pt * 16 * kDState + 32 * i + 4 * a) = S[pt][i][a];
}

// The states that the segments of a sequence start from, in place of what each
// adds: four values of a state per thread, segment after segment.
__global__ __launch_bounds__(256) void segment_kernel(KPrefill p) {
  constexpr int kBlocks = kHeadValues / 1024;
  const int part = blockIdx.x % kBlocks, h = blockIdx.x / kBlocks % p.H, seq = blockIdx.x / kBlocks / p.H;
  int b0, b1;
  if (!seq_rows(p, seq, b0, b1)) return;
  const int nseg = segments_of(p, b1 - b0);
  if (nseg < 2) return;
  const int64_t e = (int64_t)h * kHeadValues + part * 1024 + threadIdx.x * 4, slot0 = first_slot(p, seq, threadIdx.x & 63);
  if (slot0 + nseg > prefill_slots(p.rows, p.n, p.seg)) return;  // (sequences that overlap have more segments than there are slots)
  f32x4 S = p.h0 ? *reinterpret_cast<const f32x4 *>(p.h0 + (int64_t)seq * p.H * kHeadValues + e) : f32x4{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < nseg; ++i) {
    float *at = p.ws + (slot0 + i) * p.H * kHeadValues + e;
    if (i + 1 < nseg) {
      const f32x4 add = *reinterpret_cast<const f32x4 *>(at);
      const float d = exp2_d(p.decay[(slot0 + i) * p.H + h]);
      *reinterpret_cast<f32x4 *>(at) = S;
#pragma unroll
      for (int r = 0; r < 4; ++r) S[r] = fmaf(d, S[r], add[r]);
    } else {
      *reinterpret_cast<f32x4 *>(at) = S;
    }
  }
}

template <int HPW, int CT>
hipError_t prefill_t(const KPrefill &p, int out_type, hipStream_t st) {
  const int htiles = p.G * ((p.hpg + HPW - 1) / HPW);
  const int64_t ntiles = prefill_slots(p.rows, p.n, p.seg) * htiles;
  const int per_group = htiles / p.G, unit = per_group % 4 == 0 ? 4 : per_group % 2 == 0 ? 2 : 1;
  const dim3 grid((unsigned)((ntiles + 8 * unit - 1) / (8 * unit) * (8 * unit))), block(HPW * head_waves(CT) * 64);
  if (p.rows > 2 * (int64_t)p.seg) {  // a sequence may have two
    prefill_kernel<kOutF32, HPW, CT, true, false><<<grid, block, 0, st>>>(p, htiles, unit, ntiles);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    segment_kernel<<<dim3((unsigned)((int64_t)p.n * p.H * (kHeadValues / 1024))), dim3(256), 0, st>>>(p);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (out_type == kOutF32 && p.z)
    prefill_kernel<kOutF32, HPW, CT, false, true><<<grid, block, 0, st>>>(p, htiles, unit, ntiles);
  else if (out_type == kOutF32)
    prefill_kernel<kOutF32, HPW, CT, false, false><<<grid, block, 0, st>>>(p, htiles, unit, ntiles);
  else if (p.z)
    prefill_kernel<kOutBF16, HPW, CT, false, true><<<grid, block, 0, st>>>(p, htiles, unit, ntiles);
  else
    prefill_kernel<kOutBF16, HPW, CT, false, false><<<grid, block, 0, st>>>(p, htiles, unit, ntiles);
  return hipGetLastError();
}

}  // namespace

// Tokens of a segment: as many as leave two workgroups of two heads to each CU, and at least so many that the pass before
// it pays: 256 where there are few workgroups (one prompt of 64 heads, 384 : 256: 2000 tokens 59 : 50 us, 4000 95 : 80), more
// otherwise (16 of 351 to 701 tokens, 32 heads, 61 : 81; 12 of them 51 : 90; 8 of them 49 : 72; 4 of them 48 either way).
int prefill_segment(int64_t rows, int64_t n, int64_t heads) {
  const int64_t pairs = (heads + 1) / 2, want = (rows * pairs + 511) / 512, least = n * pairs <= 64 ? kLeastSegment : 384;
  return (int)((std::max<int64_t>(want, least) + kPChunk - 1) / kPChunk * kPChunk);
}

// The most slots of a call of up to so many rows and sequences.
int64_t prefill_most_slots(int64_t rows, int64_t n, int64_t heads) {
  return std::min<int64_t>(rows / kLeastSegment, 512 / ((heads + 1) / 2)) + n;
}

// Two heads a workgroup, which share B, C and their products, two waves of 32 columns each; where a CU would have no more
// than one of those, and where a group has one head, a workgroup a head, four waves of 16 columns: one prompt of 500 tokens,
// 64 heads, 50 : 33 us, 12 of 351 to 701 tokens, 32 heads, 73 : 51, 16 of them (256 workgroups of two heads) 75 : 61; one of
// 4000 tokens, 64 heads (512 of them), 80 : 87.  (Workgroups of one head of two waves took 155 us for 138 with 8 prompts of
// 500 to 1000 tokens, 64 heads of 64 groups, and operands of two parts.)
hipError_t launch_prefill(const KPrefill &p, int out_type, hipStream_t st) {
  if (p.hpg < 2) return prefill_t<1, 1>(p, out_type, st);
  const int64_t each = (p.rows + p.n - 1) / p.n, segments = each <= 2 * (int64_t)p.seg ? 1 : (each + p.seg - 1) / p.seg;
  if (p.n * segments * p.G * ((p.hpg + 1) / 2) <= 256) return prefill_t<1, 1>(p, out_type, st);
  return prefill_t<2, 2>(p, out_type, st);
}

}  // namespace ssu
