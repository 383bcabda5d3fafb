// The gated delta rule over whole sequences, in chunks of 32 tokens.
//
// Two kernels.  delta_chunk_kernel, one wave per (chunk, value head), all
// chunks at once: what of a chunk does not need the state, T = (I + A)^-1 and
// the masked decayed q . k products P, written as MFMA operands in bf16 parts.
// delta_scan_kernel, one wave per (sequence, value head, 16 columns of
// dim_v), the chunks in order: with the state's columns in registers,
//   R = b (V - e^G K^ S^T),  U = T R,  O = scale e^G Q^ S^T + P U,
//   S <- e^(G_w) S + (e^(G_w - G) U)^T K^.
// The products towards the state carry 24 bits (three bf16 parts), those
// towards the bf16 outputs 16.
#include "delta_device.cuh"

namespace ssu {

namespace {

// Chunk slot of chunk `i` of sequence s: cu[s] / 32 + s + i.  A sequence never
// has more than len / 32 + 1 chunks, so the slots of two sequences differ,
// and rows / 32 + n slots hold every sequence.
__device__ __forceinline__ int chunk_base(const DPrefill &p, int s) { return max(p.cu[s], 0) / kChunk + s; }

// The last sequence whose first chunk slot is at most `slot` (-1: none).
__device__ __forceinline__ int chunk_seq(const DPrefill &p, int slot, int lane) {
  int lo = 0, hi = p.n;
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int s = lo + lane * step;
    const uint64_t in = __ballot(s < hi && chunk_base(p, s) <= slot);
    if (in == 0) return -1;
    lo += (63 - __builtin_clzll(in)) * step;
    hi = min(hi, lo + step);
    if (step == 1) return lo;
  }
}

// [b0, b1) of sequence s; false where cu_seqlens is not what it has to be.
__device__ __forceinline__ bool seq_rows(const DPrefill &p, int s, int &b0, int &b1) {
  b0 = p.cu[s];
  b1 = p.cu[s + 1];
  return b0 >= 0 && b0 <= b1 && b1 <= p.rows;
}

template <int DK>
__global__ __launch_bounds__(64, 2) void delta_chunk_kernel(DPrefill p) {
  __shared__ WinLds<kChunk, DK> w;
  __shared__ __align__(16) float P[kChunk * (kChunk + 4)];
  __shared__ float rq[kChunk];
  const int lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  const int h = blockIdx.x % p.Hv, slot = blockIdx.x / p.Hv, hk = h / p.hpg;
  const int seq = chunk_seq(p, slot, lane);
  int b0, b1;
  if (seq < 0 || !seq_rows(p, seq, b0, b1)) return;
  const int row0 = b0 + (slot - chunk_base(p, seq)) * kChunk, W = min(kChunk, b1 - row0);
  if (W <= 0) return;

#pragma unroll
  for (int i = 0; i < kChunk * (DK / 8) / 64; ++i) {
    const int t = (i * 64 + lane) / (DK / 8), ch = (i * 64 + lane) % (DK / 8);
    st16(w.k + t * w.kKS + ch * 8,
         t < W ? ld16(p.k + (int64_t)(row0 + t) * p.k_stride + hk * DK + ch * 8) : u32x4{0, 0, 0, 0});
  }
  float2 gb = {0.f, 0.f};
  if (lane < W) {
    const int64_t o = (int64_t)(row0 + lane) * p.Hv + h;
    gb = delta_gate(p.dt[o], p.beta[o], p.A[h], p.dt_bias[h], p.softplus, p.sigmoid);
  }
  const double G = scan_d<kChunk>((double)gb.x, lane);
  if (lane < kChunk) {
    w.G[lane] = G;
    w.b[lane] = gb.y;
  }
  wave_sync();

  f32x4 kk[3], qk[3], qq[2];
  gram_kk<kChunk, DK>(w, lane, kk);
#pragma unroll
  for (int i = 0; i < 3; ++i) qk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  qq[0] = qq[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < DK / 32; ++u) {
    bf16x8 f[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int i = 16 * t + m;
      u32x4 v = {0, 0, 0, 0};
      if (i < W) v = ld16(p.q + (int64_t)(row0 + i) * p.q_stride + hk * DK + (4 * u + q) * 8);
      f[t] = __builtin_bit_cast(bf16x8, v);
      qq[t] = mfma_bf16(f[t], f[t], qq[t]);
    }
#pragma unroll
    for (int tj = 0; tj < 2; ++tj) {
      const bf16x8 kf = __builtin_bit_cast(bf16x8, ld16(w.k + (16 * tj + m) * w.kKS + (4 * u + q) * 8));
#pragma unroll
      for (int ti = tj; ti < 2; ++ti) qk[ti * (ti + 1) / 2 + tj] = mfma_bf16(f[ti], kf, qk[ti * (ti + 1) / 2 + tj]);
    }
  }
  if ((m >> 2) == q) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      w.rk[16 * t + m] = unit_of(kk[t * (t + 3) / 2], m, p.norm);
      rq[16 * t + m] = p.scale * unit_of(qq[t], m, p.norm);
    }
  }
  wave_sync();
  write_A<kChunk, DK>(w, lane, kk);
#pragma unroll
  for (int ti = 0; ti < 2; ++ti)
#pragma unroll
    for (int tj = 0; tj < 2; ++tj) {
      const int j = 16 * tj + m;
      const double Gj = w.G[j];
      const float rj = w.rk[j];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * ti + 4 * q + r;
        float v = 0.f;
        if (tj <= ti && j <= i) v = rq[i] * rj * expf((float)(w.G[i] - Gj)) * qk[tj <= ti ? ti * (ti + 1) / 2 + tj : 0][r];
        P[i * (kChunk + 4) + j] = v;
      }
    }
  wave_sync();
  invert_diag<kChunk, DK>(w, lane);

  uint8_t *rec = p.ws + ((int64_t)slot * p.Hv + h) * kRecBytes;
#pragma unroll
  for (int ti = 0; ti < 2; ++ti) {
    float x[8];
    bf16x8 f3[3], f2[2];
    t_row<kChunk, DK>(w, ti, m, q, x);
    split<3>(x, f3);
#pragma unroll
    for (int a = 0; a < 3; ++a) st16(rec + ((ti * 3 + a) * 64 + lane) * 16, __builtin_bit_cast(u32x4, f3[a]));
    depth_row<kChunk>(P + (16 * ti + m) * (kChunk + 4), q, x);
    split<2>(x, f2);
#pragma unroll
    for (int a = 0; a < 2; ++a) st16(rec + kRecT + ((ti * 2 + a) * 64 + lane) * 16, __builtin_bit_cast(u32x4, f2[a]));
  }
  float *f = reinterpret_cast<float *>(rec + kRecT + kRecP);
  if (lane < kChunk) {
    const double Gw = w.G[kChunk - 1];
    const float e = expf((float)G), rk = w.rk[lane];
    f[lane] = gb.y;
    f[32 + lane] = gb.y * e * rk;
    f[64 + lane] = expf((float)(Gw - G)) * rk;
    f[96 + lane] = rq[lane] * e;
    if (lane == 0) f[128] = expf((float)Gw);
  }
}

constexpr int kScanWaves = 4;

template <int OT, int DK>
__global__ __launch_bounds__(kScanWaves * 64) void delta_scan_kernel(DPrefill p, int groups) {
  constexpr int KS = DK + 8, VS = kScanWaves * 16 + 8, NT = DK / 16, NK = DK / 32;
  __shared__ __align__(16) uint16_t lk[kChunk * KS], lq[kChunk * KS], lv[kChunk * VS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
  const int cg = blockIdx.x % groups, h = blockIdx.x / groups % p.Hv, seq = blockIdx.x / groups / p.Hv, hk = h / p.hpg;
  int b0, b1;
  if (!seq_rows(p, seq, b0, b1)) {
    if (p.status && cg == 0 && h == 0 && tid == 0) atomicOr(p.status, SSU_STATUS_BAD_SEQLEN);
    return;
  }
  const int c0 = cg * kScanWaves * 16, col = c0 + wave * 16;  // first column of the group, of the wave
  const bool on = col < p.dv;

  f32x4 S[NT];  // rows n = 16 t + 4 q + r of the column m
  const int64_t state = (((int64_t)seq * p.Hv + h) * p.dv + col + m) * DK + 4 * q;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    S[t] = on && p.h0 ? *reinterpret_cast<const f32x4 *>(p.h0 + state + 16 * t) : f32x4{0.f, 0.f, 0.f, 0.f};

  const int first = chunk_base(p, seq);
  for (int c = 0, row0 = b0; row0 < b1; ++c, row0 += kChunk) {
    const int W = min(kChunk, b1 - row0);
    __syncthreads();  // the chunk before has been read
    for (int i = tid; i < kChunk * (DK / 8); i += kScanWaves * 64) {
      const int t = i / (DK / 8), ch = i % (DK / 8);
      u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      if (t < W) {
        a = ld16(p.k + (int64_t)(row0 + t) * p.k_stride + hk * DK + ch * 8);
        b = ld16(p.q + (int64_t)(row0 + t) * p.q_stride + hk * DK + ch * 8);
      }
      st16(lk + t * KS + ch * 8, a);
      st16(lq + t * KS + ch * 8, b);
    }
    for (int i = tid; i < kChunk * (kScanWaves * 2); i += kScanWaves * 64) {
      const int t = i / (kScanWaves * 2), ch = i % (kScanWaves * 2);
      u32x4 a = {0, 0, 0, 0};
      if (t < W && c0 + ch * 8 < p.dv) a = ld16(p.v + (int64_t)(row0 + t) * p.v_stride + h * p.dv + c0 + ch * 8);
      st16(lv + t * VS + ch * 8, a);
    }
    __syncthreads();
    if (!on) continue;

    const uint8_t *rec = p.ws + ((int64_t)(first + c) * p.Hv + h) * kRecBytes;
    const float *fac = reinterpret_cast<const float *>(rec + kRecT + kRecP);

    bf16x8 fs[NK][3];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = S[2 * ks + i / 4][i % 4];
      split<3>(x, fs[ks]);
    }

    // R = b V - (b e^G / |k|) K S^T, and O = (scale e^G / |q|) Q S^T transposed
    f32x4 o[2];
    float R[8];
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
      f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        const int at = (16 * ti + m) * KS + 32 * ks + 4 * q;
        struct { u32x2 a, b; } fk = {ld8(lk + at), ld8(lk + at + 16)}, fq = {ld8(lq + at), ld8(lq + at + 16)};
        const bf16x8 k1[1] = {__builtin_bit_cast(bf16x8, fk)}, q1[1] = {__builtin_bit_cast(bf16x8, fq)};
        x = mfma_parts(k1, fs[ks], x);
        y = mfma_bf16(fs[ks][1], q1[0], y);
        y = mfma_bf16(fs[ks][0], q1[0], y);
      }
      const f32x4 b = *reinterpret_cast<const f32x4 *>(fac + 16 * ti + 4 * q);
      const f32x4 be = *reinterpret_cast<const f32x4 *>(fac + 32 + 16 * ti + 4 * q);
      const s16x4 v = lds_tr4(lv + (16 * ti + 4 * q + (m >> 2)) * VS + wave * 16 + 4 * (m & 3));
#pragma unroll
      for (int r = 0; r < 4; ++r) R[4 * ti + r] = b[r] * bf2f((uint16_t)v[r]) - be[r] * x[r];
      o[ti] = scale4(y, fac[96 + 16 * ti + m]);
    }
    bf16x8 fr[3];
    split<3>(R, fr);
    float U[8], Ue[8];
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
      bf16x8 T[3];
#pragma unroll
      for (int a = 0; a < 3; ++a) T[a] = __builtin_bit_cast(bf16x8, ld16(rec + ((ti * 3 + a) * 64 + lane) * 16));
      const f32x4 u = mfma_parts(T, fr, f32x4{0.f, 0.f, 0.f, 0.f});
      const f32x4 e = *reinterpret_cast<const f32x4 *>(fac + 64 + 16 * ti + 4 * q);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        U[4 * ti + r] = u[r];
        Ue[4 * ti + r] = u[r] * e[r];
      }
    }
    bf16x8 fu[2], fe[3];
    split<2>(U, fu);
    split<3>(Ue, fe);
#pragma unroll
    for (int ti = 0; ti < 2; ++ti) {
      bf16x8 f[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) f[a] = __builtin_bit_cast(bf16x8, ld16(rec + kRecT + ((ti * 2 + a) * 64 + lane) * 16));
      o[ti] = mfma_parts(fu, f, o[ti]);
      if (16 * ti + m < W) {
        const int64_t at = ((int64_t)(row0 + 16 * ti + m) * p.Hv + h) * p.dv + col + 4 * q;
        if constexpr (OT == kOutF32)
          st16(static_cast<float *>(p.out) + at, __builtin_bit_cast(u32x4, o[ti]));
        else
          st8(static_cast<uint16_t *>(p.out) + at, u32x2{pack_bf16(o[ti][0], o[ti][1]), pack_bf16(o[ti][2], o[ti][3])});
      }
    }
    const float ew = fac[128];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      S[t] = Tok<32>::exact<true>(Tok<32>::load_tr(lk, KS, 16 * t, lane), fe, scale4(S[t], ew));
    }
  }
  if (on && p.h1) {
#pragma unroll
    for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(p.h1 + state + 16 * t) = S[t];
  }
}

template <int DK>
hipError_t prefill_dk(const DPrefill &p, int out_type, hipStream_t st) {
  const int64_t chunks = (int64_t)p.rows / kChunk + p.n;
  delta_chunk_kernel<DK><<<dim3((unsigned)(chunks * p.Hv)), dim3(64), 0, st>>>(p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int groups = (p.dv + kScanWaves * 16 - 1) / (kScanWaves * 16);
  const dim3 grid((unsigned)((int64_t)p.n * p.Hv * groups)), block(kScanWaves * 64);
  if (out_type == kOutF32)
    delta_scan_kernel<kOutF32, DK><<<grid, block, 0, st>>>(p, groups);
  else
    delta_scan_kernel<kOutBF16, DK><<<grid, block, 0, st>>>(p, groups);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_prefill(const DPrefill &p, int out_type, hipStream_t st) {
  return p.dk == 64 ? prefill_dk<64>(p, out_type, st) : prefill_dk<128>(p, out_type, st);
}

}  // namespace ssu
