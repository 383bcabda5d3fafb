// The selective state update over whole sequences, in chunks of 64 tokens.
//
// With G_t the running sum of A dt' within a chunk (fp64, in units of ln 2),
//   y_t = e^(G_t) C_t.S + sum_(s <= t) W_ts x_s,
//   W_ts = e^(G_t - G_s) dt'_s (C_t.B_s), + D on the diagonal,
//   S' = e^(G_w) S + sum_s (e^(G_w - G_s) dt'_s x_s) B_s^T.
// C.B is shared by the heads of a group.  A workgroup takes HPW heads of a
// group, two waves a head: 32 of its 64 columns each, their state in registers
// as matrix results [n][p], which are the next product's operand as they lie.
// B, C and x of a chunk lie in LDS, the next chunk's on their way.
//
// Long sequences are cut into segments: prefill_kernel<.., true> forms what each
// segment but the last adds to the state and its decay, segment_kernel the state that
// each starts from, then all segments run at once.
#include <algorithm>

#include "delta_device.cuh"
#include "prefill_internal.h"

namespace ssu {

namespace {

constexpr int kT = kPChunk / 16;              // token tiles of a chunk
constexpr int kTiles = kT * (kT + 1) / 2;     // C.B tiles on and below the diagonal
constexpr int kHeadValues = kHeadDim * kDState;
constexpr int BS = kDState + 8, XS = kHeadDim + 8;  // row strides in LDS: 16 rows start in different banks

constexpr int out_parts(int OT) { return OT == kOutF32 ? 3 : 2; }

__device__ __forceinline__ int slot_base(const KPrefill &p, int s) { return max(p.cu[s], 0) / p.seg + s; }

// The last sequence whose first segment slot is at most `slot` (-1: none).
__device__ __forceinline__ int slot_seq(const KPrefill &p, int slot, int lane) {
  int lo = 0, hi = p.n;
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int64_t s = lo + (int64_t)lane * step;
    const uint64_t in = __ballot(s < hi && slot_base(p, (int)min(s, (int64_t)p.n - 1)) <= slot);
    if (in == 0) return -1;
    lo += (63 - __builtin_clzll(in)) * step;
    hi = min(hi, lo + step);
    if (step == 1) return lo;
  }
}

// [b0, b1) of sequence s; false where cu_seqlens is not what it has to be.
__device__ __forceinline__ bool seq_rows(const KPrefill &p, int s, int &b0, int &b1) {
  b0 = p.cu[s];
  b1 = p.cu[s + 1];
  return b0 >= 0 && b0 <= b1 && b1 <= p.rows;
}

// What a head's tokens of a chunk contribute, in LDS.
struct Gates {
  float hi[kPChunk], lo[kPChunk];  // G in two parts: hi_t - hi_s + (lo_t - lo_s) keeps fp32 accuracy of the difference
  float dt[kPChunk], w[kPChunk], e[kPChunk];  // dt', e^(G_w - G) dt', e^G
  float last[4];                   // e^(G_w)
};

template <int HPW>
struct PBuf {
  __align__(16) uint16_t B[kPChunk * BS], C[kPChunk * BS], x[HPW][kPChunk * XS];
};

// Sums of the lanes up to and with this one.
__device__ __forceinline__ double scan64(double v, int lane) {
  v += row_shr_d<1>(v);
  v += row_shr_d<2>(v);
  v += row_shr_d<4>(v);
  v += row_shr_d<8>(v);
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  double r[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 16 * i + 15);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 16 * i + 15);
    r[i] = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  }
  if (lane >= 16) v += r[0];
  if (lane >= 32) v += r[1];
  if (lane >= 48) v += r[2];
  return v;
}
__device__ __forceinline__ double last_lane_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// By a wave: the gates of a chunk's tokens (lane = token, `there` where there is one); the whole decay's log2.
template <bool STATE>
__device__ __forceinline__ double write_gates(Gates &g, float dt, float bias, float A, int softplus, bool there, int lane) {
  const float v = dt + bias;
  const float d = there ? (softplus ? softplus_f(v) : v) : 0.f;
  double a = (double)A * d;
  a = there ? (a < -0x1p20 ? -0x1p20 : a) : 0.0;  // (NaN stays)
  const double G = scan64(a * kLog2e, lane), Gw = last_lane_d(G);
  if constexpr (!STATE) {
    const float hi = (float)G;
    g.hi[lane] = hi;
    g.lo[lane] = (float)(G - (double)hi);
    g.dt[lane] = d;
    g.e[lane] = exp2_d(G);
  }
  g.w[lane] = exp2_d(Gw - G) * d;
  if (lane == 0) g.last[0] = exp2_d(Gw);
  return Gw;
}

__device__ __forceinline__ bf16x8 row_frag(const uint16_t *rows, int stride, int t0, int n0, int lane) {
  return __builtin_bit_cast(bf16x8, ld16(rows + (t0 + (lane & 15)) * stride + n0 + 8 * (lane >> 4)));
}

// A chunk's rows on their way from memory to LDS through the registers of NT
// threads; rows behind the segment's last repeat it (their dt' is 0), heads
// behind the group's last repeat that.  Every load is unconditional.
template <int HPW, bool STATE>
struct PStage {
  static constexpr int NT = HPW * 128, NB = kPChunk * kDState / 8 / NT, NX = kPChunk * kHeadDim / 8 / 128;
  u32x4 b[NB], c[STATE ? 1 : NB], x[NX];

  __device__ __forceinline__ void fetch(const KPrefill &p, int64_t row0, int last, int g, int h0, int heads, int tid) {
    const char *Bp = reinterpret_cast<const char *>(p.B + row0 * p.B_stride + g * kDState);
    const char *Cp = reinterpret_cast<const char *>(p.C + row0 * p.C_stride + g * kDState);
    const char *xp = reinterpret_cast<const char *>(p.x + row0 * p.x_stride + h0 * kHeadDim);
    const uint32_t bs = (uint32_t)p.B_stride * 2, cs = (uint32_t)p.C_stride * 2, xs = (uint32_t)p.x_stride * 2;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int at = i * NT + tid, t = min(at / (kDState / 8), last), ch = at % (kDState / 8);
      b[i] = ld16(Bp + (uint32_t)t * bs + ch * 16);
      if constexpr (!STATE) c[i] = ld16(Cp + (uint32_t)t * cs + ch * 16);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int at = i * NT + tid, t = min(at / (HPW * 8), last), ch = at % (HPW * 8), hh = min(ch / 8, heads - 1);
      x[i] = ld16(xp + (uint32_t)t * xs + hh * 128 + ch % 8 * 16);
    }
  }
  __device__ __forceinline__ void store(PBuf<HPW> &o, int tid) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int at = i * NT + tid, t = at / (kDState / 8), ch = at % (kDState / 8);
      st16(o.B + t * BS + ch * 8, b[i]);
      if constexpr (!STATE) st16(o.C + t * BS + ch * 8, c[i]);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int at = i * NT + tid, t = at / (HPW * 8), ch = at % (HPW * 8);
      st16(o.x[ch / 8] + t * XS + ch % 8 * 8, x[i]);
    }
  }
};

// Lane (m, q) of a wave holds of the state column p = p0 + 16 pt + m, values n =
// 32 i + 8 q + 4 a + r in S[pt][i][a][r]; of the outputs row p0 + 16 pt + 4 q + r,
// token 16 ti + m in y[pt][ti][r].
template <int OT, int HPW, bool STATE>
__global__ __launch_bounds__(HPW * 128) void prefill_kernel(KPrefill p, int htiles, int64_t ntiles) {
  constexpr int NP = out_parts(OT);
  __shared__ PBuf<HPW> buf[2];
  __shared__ Gates gates[HPW];
  __shared__ f32x4 cb[STATE ? 1 : kTiles][64];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), hh = wave >> 1, p0 = (wave & 1) * 32;
  if (!STATE) {
    for (int64_t s = (int64_t)blockIdx.x * (HPW * 128) + tid; s < p.n; s += (int64_t)gridDim.x * (HPW * 128)) {
      int b0, b1;
      if (!seq_rows(p, (int)s, b0, b1) && p.status) atomicOr(p.status, SSU_STATUS_BAD_SEQLEN);
    }
  }
  const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
  if (tile >= ntiles) return;
  const int per_group = htiles / p.G;
  const int ht = (int)(tile % htiles), slot = (int)(tile / htiles);
  const int g = ht / per_group, hfirst = g * p.hpg + ht % per_group * HPW, heads = min(HPW, (g + 1) * p.hpg - hfirst);
  const int seq = slot_seq(p, slot, lane);
  int b0, b1;
  if (seq < 0 || !seq_rows(p, seq, b0, b1)) return;
  const int i_seg = slot - slot_base(p, seq), nseg = max(1, (int)(((int64_t)b1 - b0 + p.seg - 1) / p.seg));
  if (i_seg >= (STATE ? nseg - 1 : nseg)) return;
  const int64_t row0 = b0 + (int64_t)i_seg * p.seg;
  const int rows = (int)min((int64_t)p.seg, b1 - row0), chunks = (rows + kPChunk - 1) / kPChunk;
  const bool on = hh < heads;
  const int h = hfirst + min(hh, heads - 1);

  f32x4 S[2][4][2];
  const int64_t own = (int64_t)h * kHeadValues + (p0 + m) * kDState + 8 * q;  // of (i, a, pt) = 0
  const float *from = STATE ? nullptr : (nseg > 1 ? p.ws + (int64_t)slot * p.H * kHeadValues : p.h0 ? p.h0 + (int64_t)seq * p.H * kHeadValues : nullptr);
#pragma unroll
  for (int pt = 0; pt < 2; ++pt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int a = 0; a < 2; ++a)
        S[pt][i][a] = from ? *reinterpret_cast<const f32x4 *>(from + own + pt * 16 * kDState + 32 * i + 4 * a) : f32x4{0.f, 0.f, 0.f, 0.f};

  if (chunks > 0) {
    const float A = p.A[h], bias = p.dt_bias[h], D = STATE ? 0.f : p.D[h];
    double total = 0.0;
    PStage<HPW, STATE> st;
    auto last_of = [&](int c) { return min(kPChunk, rows - c * kPChunk) - 1; };
    auto dt_of = [&](int c) { return p.dt[(row0 + c * kPChunk + min(lane, last_of(c))) * p.H + h]; };
    st.fetch(p, row0, last_of(0), g, hfirst, heads, tid);
    float dt = dt_of(0);
    st.store(buf[0], tid);
    for (int c = 0; c < chunks; ++c) {
      const PBuf<HPW> &in = buf[c & 1];
      const int W = last_of(c) + 1, next = min(c + 1, chunks - 1);
      const int64_t r0 = row0 + c * kPChunk;
      __syncthreads();
      st.fetch(p, row0 + (int64_t)next * kPChunk, last_of(next), g, hfirst, heads, tid);
      if ((wave & 1) == 0) total += write_gates<STATE>(gates[hh], dt, bias, A, p.softplus, lane < W, lane);
      dt = dt_of(next);
      if constexpr (!STATE) {
#pragma unroll
        for (int k = 0; k < (kTiles + 2 * HPW - 1) / (2 * HPW); ++k) {
          const int tile_at = k * 2 * HPW + wave;
          if (tile_at < kTiles) {
            const int ti = tile_at >= 6 ? 3 : tile_at >= 3 ? 2 : tile_at >= 1 ? 1 : 0, si = tile_at - ti * (ti + 1) / 2;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < 4; ++u)
              v = mfma_bf16(row_frag(in.B, BS, 16 * si, 32 * u, lane), row_frag(in.C, BS, 16 * ti, 32 * u, lane), v);
            cb[tile_at][lane] = v;
          }
        }
      }
      __syncthreads();
      const Gates &gt = gates[hh];
      const uint16_t *x = in.x[hh];
      bf16x8 xf[2][2];
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) xf[pt][ks] = Tok<32>::load_tr(x + 32 * ks * XS, XS, p0 + 16 * pt, lane);
      if constexpr (!STATE) {
        f32x4 y[2][kT];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int ti = 0; ti < kT; ++ti) y[pt][ti] = f32x4{0.f, 0.f, 0.f, 0.f};
        // the state's readout
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bf16x8 f[2][NP];
#pragma unroll
          for (int pt = 0; pt < 2; ++pt) {
            const float v[8] = {S[pt][i][0][0], S[pt][i][0][1], S[pt][i][0][2], S[pt][i][0][3],
                                S[pt][i][1][0], S[pt][i][1][1], S[pt][i][1][2], S[pt][i][1][3]};
            split<NP>(v, f[pt]);
          }
#pragma unroll
          for (int ti = 0; ti < kT; ++ti) {
            const bf16x8 cf = row_frag(in.C, BS, 16 * ti, 32 * i, lane);
#pragma unroll
            for (int a = NP - 1; a >= 0; --a)
#pragma unroll
              for (int pt = 0; pt < 2; ++pt) y[pt][ti] = mfma_bf16(f[pt][a], cf, y[pt][ti]);
          }
        }
        // the tokens of the chunk, and out
#pragma unroll
        for (int ti = 0; ti < kT; ++ti) {
          const int t = 16 * ti + m;
          const float e = gt.e[t], hi = gt.hi[t], lo = gt.lo[t];
#pragma unroll
          for (int pt = 0; pt < 2; ++pt) y[pt][ti] = scale4(y[pt][ti], e);
#pragma unroll
          for (int ks = 0; ks <= ti / 2; ++ks) {
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
              const f32x4 shi = *reinterpret_cast<const f32x4 *>(gt.hi + s0), slo = *reinterpret_cast<const f32x4 *>(gt.lo + s0);
              const f32x4 sdt = *reinterpret_cast<const f32x4 *>(gt.dt + s0);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float d = __builtin_amdgcn_exp2f((hi - shi[r]) + (lo - slo[r])) * sdt[r] * v[r];
                w[4 * a + r] = si < ti || s0 + r < t ? d : (s0 + r == t ? d + D : 0.f);
              }
            }
            bf16x8 wf[NP];
            split<NP>(w, wf);
#pragma unroll
            for (int a = NP - 1; a >= 0; --a)
#pragma unroll
              for (int pt = 0; pt < 2; ++pt) y[pt][ti] = mfma_bf16(xf[pt][ks], wf[a], y[pt][ti]);
          }
          if (on && t < W) {
#pragma unroll
            for (int pt = 0; pt < 2; ++pt) {
              const int col = h * kHeadDim + p0 + 16 * pt + 4 * q;
              f32x4 v = y[pt][ti];
              if (p.z) {
                const u32x2 zw = ld8(p.z + (r0 + t) * p.z_stride + col);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float z = bf2f((zw[r >> 1] >> (16 * (r & 1))) & 0xFFFFu);
                  v[r] = v[r] * z / (1.f + expf(-z));
                }
              }
              const int64_t at = (r0 + t) * p.H * kHeadDim + col;
              if constexpr (OT == kOutF32)
                *reinterpret_cast<f32x4 *>(static_cast<float *>(p.out) + at) = v;
              else
                st8(static_cast<uint16_t *>(p.out) + at, u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])});
            }
          }
        }
      }
      // S <- e^(G_w) S + B^T (w x)
      bf16x8 xw[2][2][3];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const f32x4 w0 = *reinterpret_cast<const f32x4 *>(gt.w + 32 * ks + 4 * q);
        const f32x4 w1 = *reinterpret_cast<const f32x4 *>(gt.w + 32 * ks + 16 + 4 * q);
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) {
          const u32x4 xx = __builtin_bit_cast(u32x4, xf[pt][ks]);
          float v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = bf2f((xx[r >> 1] >> (16 * (r & 1))) & 0xFFFFu) * (r < 4 ? w0[r & 3] : w1[r & 3]);
          split<3>(v, xw[pt][ks]);
        }
      }
      const float ew = gt.last[0];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
#pragma unroll
          for (int pt = 0; pt < 2; ++pt) S[pt][i][a] = scale4(S[pt][i][a], ew);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            // row m = 4 j + r of the tile is n = 32 i + 8 j + 4 a + r
            const uint16_t *at = in.B + (32 * ks + 4 * q + (m >> 2)) * BS + 32 * i + 8 * (m & 3) + 4 * a;
            struct { s16x4 lo, hi; } bt = {lds_tr4(at), lds_tr4(at + 16 * BS)};
            const bf16x8 bf = __builtin_bit_cast(bf16x8, bt);
#pragma unroll
            for (int k = 2; k >= 0; --k)
#pragma unroll
              for (int pt = 0; pt < 2; ++pt) S[pt][i][a] = mfma_bf16(bf, xw[pt][ks][k], S[pt][i][a]);
          }
        }
      st.store(buf[(c + 1) & 1], tid);
    }
    if (STATE && (wave & 1) == 0 && lane == 0 && on) p.decay[(int64_t)slot * p.H + h] = total;
  }
  float *to = STATE ? p.ws + (int64_t)slot * p.H * kHeadValues : (p.h1 && i_seg == nseg - 1 ? p.h1 + (int64_t)seq * p.H * kHeadValues : nullptr);
  if (!to || !on) return;
#pragma unroll
  for (int pt = 0; pt < 2; ++pt)
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
  const int nseg = (int)(((int64_t)b1 - b0 + p.seg - 1) / p.seg);
  if (nseg < 2) return;
  const int64_t e = (int64_t)h * kHeadValues + part * 1024 + threadIdx.x * 4, slot0 = slot_base(p, seq);
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

template <int HPW>
hipError_t prefill_hpw(const KPrefill &p, int out_type, hipStream_t st) {
  const int htiles = p.G * ((p.hpg + HPW - 1) / HPW);
  const int64_t ntiles = prefill_slots(p.rows, p.n, p.seg) * htiles;
  const dim3 grid(xcd_grid(ntiles)), block(HPW * 128);
  if (p.rows > p.seg) {
    prefill_kernel<kOutF32, HPW, true><<<grid, block, 0, st>>>(p, htiles, ntiles);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    segment_kernel<<<dim3((unsigned)((int64_t)p.n * p.H * (kHeadValues / 1024))), dim3(256), 0, st>>>(p);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (out_type == kOutF32)
    prefill_kernel<kOutF32, HPW, false><<<grid, block, 0, st>>>(p, htiles, ntiles);
  else
    prefill_kernel<kOutBF16, HPW, false><<<grid, block, 0, st>>>(p, htiles, ntiles);
  return hipGetLastError();
}

}  // namespace

// Tokens of a segment: about 1024 (segment, head) pairs, and no segment shorter than 512 tokens.
int prefill_segment(int64_t rows, int64_t n, int64_t heads) {
  (void)n;
  const int64_t want = (rows * heads + 1023) / 1024;
  return (int)(std::max<int64_t>(want, 512) + kPChunk - 1) / kPChunk * kPChunk;
}

hipError_t launch_prefill(const KPrefill &p, int out_type, hipStream_t st) {
  if (p.hpg >= 4) return prefill_hpw<4>(p, out_type, st);
  if (p.hpg >= 2) return prefill_hpw<2>(p, out_type, st);
  return prefill_hpw<1>(p, out_type, st);
}

}  // namespace ssu
