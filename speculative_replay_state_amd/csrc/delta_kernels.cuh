// The gated delta rule on cached requests: step, flush, init and read
// (one instantiation per checkpoint type).
//
// Step.  With M = P T (P_ij = scale e^(G_i - G_j) q^_i . k^_j) the outputs need
// neither U nor the state's products with k:
//   o_i = S (scale e^(G_i) q^_i - sum_j M_ij b_j e^(G_j) k^_j) + sum_j M_ij b_j v_j,
// one readout of the checkpoint with a query per new token, as in the
// selective state update.  A wave forms the queries of its (entry, head) in
// registers while its rows of the checkpoint are on their way, then reads
// them out: HBM traffic is the checkpoint once, the window and the outputs.
//
// Flush.  U = (T b) V - W S^T with W = T b e^G K^ (rows = tokens), then the
// rank-k update, both MFMA products with the checkpoint rows in registers.
#pragma once

#include "delta_device.cuh"

namespace ssu {

// 16-byte chunks of a lane per row block
constexpr int dchunks(int ST, int DK) { return DK / 4 * (ST == kF32 ? 4 : 2) / 16; }

// A row block of the checkpoint (16 rows, 16-byte chunks of a lane) as MFMA
// operands of NS parts.
template <int ST, int DK, int NS>
__device__ __forceinline__ void state_operand(const u32x4 *ch, int ks, bf16x8 (&f)[NS]) {
  if constexpr (ST == kBF16) {
    f[0] = __builtin_bit_cast(bf16x8, ch[ks]);
  } else {
    float x[8];
    if constexpr (ST == kF16) {
      const f16x8 v = __builtin_bit_cast(f16x8, ch[ks]);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(ch[2 * ks + i / 4][i % 4]);
    }
    split<NS>(x, f);
  }
}

// value i of the lane's DK / 4 as fp32
template <int ST>
__device__ __forceinline__ float state_value(const u32x4 *ch, int i) {
  if constexpr (ST == kF32) return __uint_as_float(ch[i / 4][i % 4]);
  const uint32_t w = ch[i / 8][i % 8 / 2];
  const uint16_t v = (uint16_t)(i & 1 ? w >> 16 : w);
  if constexpr (ST == kBF16) return bf2f(v);
  return (float)__builtin_bit_cast(_Float16, v);
}

template <int ST, int DK>
__device__ __forceinline__ void state_encode(const float (&x)[DK / 4], u32x4 (&ch)[dchunks(ST, DK)]) {
  constexpr int E = ST == kF32 ? 4 : 8;
#pragma unroll
  for (int u = 0; u < dchunks(ST, DK); ++u)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (ST == kF32) ch[u][w] = __float_as_uint(x[E * u + w]);
      if constexpr (ST == kBF16) ch[u][w] = pack_bf16(x[E * u + 2 * w], x[E * u + 2 * w + 1]);
      if constexpr (ST == kF16) ch[u][w] = pack_f16(x[E * u + 2 * w], x[E * u + 2 * w + 1]);
    }
}

struct DEntry {
  int slot, p, r, T, bos;
  int mode;  // 0: nothing, 1: zero output rows, 2: replay
};

__device__ __forceinline__ DEntry delta_entry(const DCache &c, const DStep &s, int b, bool report) {
  DEntry e;
  e.bos = s.cu ? s.cu[b] : b * s.T;
  e.T = s.cu ? s.cu[b + 1] - e.bos : s.T;
  e.slot = s.slot_idx[b];
  e.p = s.pnat[b];
  e.r = 0;
  e.mode = 2;
  int bit = 0;
  if (e.T < 0 || e.T > s.T || e.bos < 0) {
    e.mode = 0;
    bit = SSU_STATUS_BAD_SEQLEN;
  } else if (e.slot <= 0 || e.slot >= c.num_slots) {
    e.mode = 1;
  } else if (e.p < 0 || e.p > c.L - e.T) {
    e.mode = 1;
    bit = SSU_STATUS_BAD_PNAT;
  } else {
    e.r = c.ring_start[e.slot];
    if (e.r < 0 || e.r >= c.L) {
      e.mode = 1;
      bit = SSU_STATUS_BAD_RING;
    }
  }
  if (bit && report && c.status && threadIdx.x == 0) atomicOr(c.status, bit);
  return e;
}

constexpr int kStepWaveChunks = 16;  // 16-byte chunks of the checkpoint a lane keeps in flight

template <int ST, int OT, int KW, int DK>
__global__ __launch_bounds__(64, 2) void delta_step_kernel(DCache c, DStep s, int parts, int64_t nwaves) {
  constexpr int CH = dchunks(ST, DK), RB = kStepWaveChunks / CH, E = KW / 4;
  constexpr int NQ = OT == kOutF32 ? 3 : 2, NS = ST == kF32 ? NQ : (ST == kF16 ? 2 : 1);
  constexpr int VS = RB * 16 + 8;
  typedef typename Tok<KW>::V TV;
  constexpr int KS = DK + 8;  // row strides in LDS: 8 values on, so 16 rows start in different banks
  __shared__ WinLds<KW> w;
  __shared__ float rq[16];
  __shared__ __align__(16) uint16_t kw[KW * KS], vw[KW * VS];

  const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
  if (tile >= nwaves) return;
  const int lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  const int part = (int)(tile % parts);
  const int64_t pair = tile / parts;
  const int h = (int)(pair % c.Hv), b = (int)(pair / c.Hv), hk = h / c.hpg;
  const DEntry e = delta_entry(c, s, b, part == 0 && h == 0);
  if (e.mode == 0 || e.T == 0) return;
  const int rb0 = part * RB, nrb = min(RB, c.dv / 16 - rb0);
  if (e.mode == 1) {
    for (int i = lane; i < e.T * nrb * 4; i += 64) {
      const int t = i / (nrb * 4), ch = i % (nrb * 4);
      const int64_t o = ((int64_t)(e.bos + t) * c.Hv + h) * c.dv + rb0 * 16 + ch * 4;
      if constexpr (OT == kOutF32)
        st16(static_cast<float *>(s.out) + o, u32x4{0, 0, 0, 0});
      else
        st8(static_cast<uint16_t *>(s.out) + o, u32x2{0, 0});
    }
    return;
  }

  // the checkpoint rows, on their way while the queries are formed
  u32x4 st[RB][CH];
  {
    const uint8_t *src = c.state + (int64_t)e.slot * c.state_stride +
                         ((int64_t)h * c.dv / 16 + rb0) * (CH * 1024) + lane * 16;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int u = 0; u < CH; ++u)
        st[i][u] = i < nrb ? ld16_nt(src + (i * CH + u) * 1024) : u32x4{0, 0, 0, 0};
  }

  // the window: p live tokens of the ring, then the new ones; behind it zeros
  const int p = e.p, W = p + e.T;
  uint8_t *ring_k = c.kc + (int64_t)e.slot * c.k_stride + (int64_t)hk * c.L * DK * 2;
  uint8_t *ring_v = c.vc + (int64_t)e.slot * c.v_stride + (int64_t)h * c.L * c.dv * 2;
  float2 *ring_g = reinterpret_cast<float2 *>(c.gc + (int64_t)e.slot * c.g_stride) + (int64_t)h * c.L;
  const bool first = part == 0, first_k = first && h % c.hpg == 0;
#pragma unroll
  for (int i = 0; i < KW * (DK / 8) / 64; ++i) {
    const int t = (i * 64 + lane) / (DK / 8), ch = (i * 64 + lane) % (DK / 8);
    u32x4 v = {0, 0, 0, 0};
    if (t < W) {
      uint8_t *at = ring_k + (ring_pos(e.r, t, c.L) * DK + ch * 8) * 2;
      v = t < p ? ld16(at) : ld16(s.k + (int64_t)(e.bos + t - p) * s.k_stride + hk * DK + ch * 8);
      if (t >= p && first_k) st16(at, v);
    }
    st16(kw + t * KS + ch * 8, v);
  }
#pragma unroll
  for (int i = 0; i < (KW * RB * 2 + 63) / 64; ++i) {
    const int at = i * 64 + lane, t = at / (RB * 2), ch = at % (RB * 2);
    if (at < KW * RB * 2) {
      u32x4 v = {0, 0, 0, 0};
      if (t < W && ch < nrb * 2) {
        uint8_t *dst = ring_v + ((int64_t)ring_pos(e.r, t, c.L) * c.dv + rb0 * 16 + ch * 8) * 2;
        v = t < p ? ld16(dst) : ld16(s.v + (int64_t)(e.bos + t - p) * s.v_stride + h * c.dv + rb0 * 16 + ch * 8);
        if (t >= p) st16(dst, v);
      }
      st16(vw + t * VS + ch * 8, v);
    }
  }
  bf16x8 qn[DK / 32];
  u32x2 qd[DK / 16];
  {
    const uint16_t *qr = s.q + (int64_t)(e.bos + (m < e.T ? m : 0)) * s.q_stride + hk * DK;
#pragma unroll
    for (int u = 0; u < DK / 32; ++u) qn[u] = __builtin_bit_cast(bf16x8, ld16(qr + (4 * u + q) * 8));
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) qd[t] = ld8(qr + 16 * t + 4 * q);
  }
  float2 gb = {0.f, 0.f};
  if (lane < W) {
    float2 *at = ring_g + ring_pos(e.r, lane, c.L);
    if (lane < p) {
      gb = *at;
    } else {
      const int64_t o = (int64_t)(e.bos + lane - p) * c.Hv + h;
      gb = delta_gate(s.dt[o], s.beta[o], s.A[h], s.dt_bias[h], s.softplus, s.sigmoid);
      if (first) *at = gb;
    }
  }
  const double G = scan_d<KW>((double)gb.x * kLog2e, lane);
  if (lane < KW) {
    w.G[lane] = G;
    w.b[lane] = gb.y;
  }
  wave_sync();

  // k . k and k . q over the window, and the units from their diagonals
  f32x4 kk[win_tiles(KW)], qk[KW / 16], qq = {0.f, 0.f, 0.f, 0.f}, decay[win_tiles(KW)];
#pragma unroll
  for (int t = 0; t < win_tiles(KW); ++t) kk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < KW / 16; ++t) qk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < DK / 32; ++u) {
    bf16x8 f[KW / 16];
#pragma unroll
    for (int t = 0; t < KW / 16; ++t) {
      f[t] = __builtin_bit_cast(bf16x8, ld16(kw + (16 * t + m) * KS + (4 * u + q) * 8));
      qk[t] = mfma_bf16(f[t], qn[u], qk[t]);
    }
    qq = mfma_bf16(qn[u], qn[u], qq);
    gram_kk<KW>(f, kk);
  }
  write_rk<KW>(w, m, q, kk, c.norm);
  if ((m >> 2) == q) rq[m] = s.scale * unit_of(qq, m, c.norm);
  wave_sync();
  write_A<KW>(w, m, q, kk, decay);
  // row m of P along the tokens
  f32x4 P[KW / 16];
  const int at = p + min(m, e.T - 1);
  const double Gm = w.G[at];
  const float rqm = m < e.T ? rq[m] : 0.f;
#pragma unroll
  for (int t = 0; t < KW / 16; ++t) {
    const int j0 = 16 * t + 4 * q;
    const f32x4 rj = *reinterpret_cast<const f32x4 *>(w.rk + j0);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      P[t][r] = j0 + r <= at ? rqm * rj[r] * exp2_d(Gm - w.G[j0 + r]) * qk[t][r] : 0.f;
  }
  wave_sync();
  invert_diag<KW>(w, lane);

  // row m of M: the weights of v and (with b e^G / |k|) of k
  float cv[E], ck[E];
  m_row<KW>(w, P, m, q, cv);
#pragma unroll
  for (int a = 0; a < KW / 16; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 16 * a + 4 * q + r;
      cv[4 * a + r] *= w.b[j];
      ck[4 * a + r] = -cv[4 * a + r] * exp2_d(w.G[j]) * w.rk[j];
    }
  TV fv[NQ], fk[NQ];
  split<NQ>(cv, fv);
  split<NQ>(ck, fk);

  // the queries, one column per new token
  bf16x8 fq[DK / 32][NQ];
  {
    const float eq = rqm * exp2_d(Gm);
    float y[DK / 4];
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) {
      f32x4 acc = {eq * bf2f(qd[t][0] & 0xFFFFu), eq * __uint_as_float(qd[t][0] & 0xFFFF0000u),
                   eq * bf2f(qd[t][1] & 0xFFFFu), eq * __uint_as_float(qd[t][1] & 0xFFFF0000u)};
      acc = Tok<KW>::template exact<true>(Tok<KW>::load_tr(kw, KS, 16 * t, lane), fk, acc);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[4 * t + r] = acc[r];
    }
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = y[8 * ks + i];
      split<NQ>(z, fq[ks]);
    }
  }

#pragma unroll
  for (int i = 0; i < RB; ++i) {
    if (i >= nrb) break;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      bf16x8 f[NS];
      state_operand<ST, DK, NS>(st[i], ks, f);
      acc = mfma_parts(f, fq[ks], acc);
    }
    acc = Tok<KW>::template exact<true>(Tok<KW>::load_tr(vw, VS, 16 * i, lane), fv, acc);
    if (m < e.T) {
      const int64_t o = ((int64_t)(e.bos + m) * c.Hv + h) * c.dv + (rb0 + i) * 16 + 4 * q;
      if constexpr (OT == kOutF32)
        st16(static_cast<float *>(s.out) + o, __builtin_bit_cast(u32x4, acc));
      else
        st8(static_cast<uint16_t *>(s.out) + o, u32x2{pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3])});
    }
  }
}

// Whether slot_idx[j] folds k tokens, with the status bits of ssu_delta_flush.
__device__ __forceinline__ bool delta_fold_entry(const DCache &c, int slot, int k, int &r, bool report) {
  if (slot <= 0 || slot >= c.num_slots || k == 0) return false;
  int bit = 0;
  if (k < 0 || k > c.L) {
    bit = SSU_STATUS_BAD_FOLD;
  } else {
    r = c.ring_start[slot];
    if (r < 0 || r >= c.L) bit = SSU_STATUS_BAD_RING;
  }
  if (bit && report && c.status) atomicOr(c.status, bit);
  return bit == 0;
}

template <int ST, int KW, int DK>
__global__ __launch_bounds__(64, 2) void delta_flush_kernel(DCache c, const int32_t *slot_idx, const int32_t *num_fold,
                                                         int parts, int64_t nwaves) {
  constexpr int CH = dchunks(ST, DK), RB = kStepWaveChunks / CH, E = KW / 4, NT = KW / 16;
  constexpr int NW = ST == kF32 ? 3 : 2, NS = ST == kBF16 ? 1 : 2;
  constexpr int VS = RB * 16 + 8;
  typedef typename Tok<KW>::V TV;
  constexpr int KS = DK + 8;
  __shared__ WinLds<KW> w;
  __shared__ __align__(16) uint16_t kw[KW * KS], vw[KW * VS];

  const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
  if (tile >= nwaves) return;
  const int lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  const int part = (int)(tile % parts);
  const int64_t pair = tile / parts;
  const int h = (int)(pair % c.Hv), b = (int)(pair / c.Hv), hk = h / c.hpg;
  const int slot = slot_idx[b], k = num_fold[b];
  int ring = 0;
  if (!delta_fold_entry(c, slot, k, ring, part == 0 && h == 0 && lane == 0)) return;
  const int rb0 = part * RB, nrb = min(RB, c.dv / 16 - rb0);

  uint8_t *tiles = c.state + (int64_t)slot * c.state_stride + ((int64_t)h * c.dv / 16 + rb0) * (CH * 1024) + lane * 16;
  u32x4 st[RB][CH];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int u = 0; u < CH; ++u) st[i][u] = i < nrb ? ld16_nt(tiles + (i * CH + u) * 1024) : u32x4{0, 0, 0, 0};

  const uint8_t *ring_k = c.kc + (int64_t)slot * c.k_stride + (int64_t)hk * c.L * DK * 2;
  const uint8_t *ring_v = c.vc + (int64_t)slot * c.v_stride + (int64_t)h * c.L * c.dv * 2;
  const float2 *ring_g = reinterpret_cast<const float2 *>(c.gc + (int64_t)slot * c.g_stride) + (int64_t)h * c.L;
#pragma unroll
  for (int i = 0; i < KW * (DK / 8) / 64; ++i) {
    const int t = (i * 64 + lane) / (DK / 8), ch = (i * 64 + lane) % (DK / 8);
    st16(kw + t * KS + ch * 8,
         t < k ? ld16(ring_k + (ring_pos(ring, t, c.L) * DK + ch * 8) * 2) : u32x4{0, 0, 0, 0});
  }
#pragma unroll
  for (int i = 0; i < (KW * RB * 2 + 63) / 64; ++i) {
    const int at = i * 64 + lane, t = at / (RB * 2), ch = at % (RB * 2);
    if (at < KW * RB * 2)
      st16(vw + t * VS + ch * 8, t < k && ch < nrb * 2
                                     ? ld16(ring_v + ((int64_t)ring_pos(ring, t, c.L) * c.dv + rb0 * 16 + ch * 8) * 2)
                                     : u32x4{0, 0, 0, 0});
  }
  const float2 gb = lane < k ? ring_g[ring_pos(ring, lane, c.L)] : float2{0.f, 0.f};
  const double G = scan_d<KW>((double)gb.x * kLog2e, lane);
  if (lane < KW) {
    w.G[lane] = G;
    w.b[lane] = gb.y;
  }
  wave_sync();
  {
    f32x4 kk[win_tiles(KW)], decay[win_tiles(KW)];
#pragma unroll
    for (int t = 0; t < win_tiles(KW); ++t) kk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < DK / 32; ++u) {
      bf16x8 f[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) f[t] = __builtin_bit_cast(bf16x8, ld16(kw + (16 * t + m) * KS + (4 * u + q) * 8));
      gram_kk<KW>(f, kk);
    }
    write_rk<KW>(w, m, q, kk, c.norm);
    wave_sync();
    write_A<KW>(w, m, q, kk, decay);
  }
  wave_sync();
  invert_diag<KW>(w, lane);

  // T b (towards V) and W = T b e^G K^ as operands, rows = tokens
  TV ft[NT][NW], kt[DK / 16];
  bf16x8 fw[NT][DK / 32][2];
#pragma unroll
  for (int t = 0; t < DK / 16; ++t) kt[t] = Tok<KW>::load_tr(kw, KS, 16 * t, lane);
  float bj[E], ej[E];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 16 * a + 4 * q + r;
      bj[4 * a + r] = w.b[j];
      ej[4 * a + r] = -exp2_d(w.G[j]) * w.rk[j];
    }
#pragma unroll
  for (int ti = 0; ti < NT; ++ti) {
    float x[E], y[E];
    t_row<KW>(w, ti, m, q, x);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x[i] *= bj[i];
      y[i] = x[i] * ej[i];
    }
    split<NW>(x, ft[ti]);
    TV fy[NW];
    split<NW>(y, fy);
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      float z[8];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const f32x4 acc = Tok<KW>::template exact<true>(kt[2 * ks + a], fy, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int r = 0; r < 4; ++r) z[4 * a + r] = acc[r];
      }
      split<2>(z, fw[ti][ks]);
    }
  }
  const double Gw = w.G[KW - 1];
  const float ew = exp2_d(Gw);
  float fu[E];  // e^(G_w - G_i) / |k_i| of the lane's rows
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 16 * a + 4 * q + r;
      fu[4 * a + r] = exp2_d(Gw - w.G[j]) * w.rk[j];
    }

#pragma unroll
  for (int i = 0; i < RB; ++i) {
    if (i >= nrb) break;
    bf16x8 f[DK / 32][NS];
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) state_operand<ST, DK, NS>(st[i], ks, f[ks]);
    const TV vt = Tok<KW>::load_tr(vw, VS, 16 * i, lane);
    float u[E];
#pragma unroll
    for (int ti = 0; ti < NT; ++ti) {
      f32x4 acc = Tok<KW>::template exact<false>(vt, ft[ti], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) acc = mfma_parts(fw[ti][ks], f[ks], acc);
#pragma unroll
      for (int r = 0; r < 4; ++r) u[4 * ti + r] = acc[r] * fu[4 * ti + r];
    }
    TV fuu[NW];
    split<NW>(u, fuu);
    float y[DK / 4];
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) {
      f32x4 acc;
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = ew * state_value<ST>(st[i], 4 * t + r);
      acc = Tok<KW>::template exact<true>(kt[t], fuu, acc);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[4 * t + r] = acc[r];
    }
    u32x4 o[CH];
    state_encode<ST, DK>(y, o);
#pragma unroll
    for (int v = 0; v < CH; ++v) st16_nt(tiles + (i * CH + v) * 1024, o[v]);
  }
}

template <int ST>  // one instantiation, and one symbol, per checkpoint type's object
__global__ void delta_ring_advance_kernel(DCache c, const int32_t *slot_idx, const int32_t *num_fold, int n) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= n) return;
  const int slot = slot_idx[j], k = num_fold[j];
  int r = 0;
  if (delta_fold_entry(c, slot, k, r, false)) c.ring_start[slot] = ring_pos(r, k, c.L);
}

// fp32 row-major states to (READ: from) the checkpoints: a wave per row block,
// four values of a row per lane and step.
template <int ST, int DK, bool READ>
__global__ __launch_bounds__(64) void delta_state_kernel(DCache c, float *states, int64_t stride,
                                                         const int32_t *slot_idx, int64_t nwaves) {
  constexpr int CH = dchunks(ST, DK);
  const int64_t tile = blockIdx.x;
  if (tile >= nwaves) return;
  const int nrb = c.dv / 16, lane = threadIdx.x, m = lane & 15, q = lane >> 4;
  const int rb = (int)(tile % nrb), h = (int)(tile / nrb % c.Hv);
  const int64_t j = tile / nrb / c.Hv;
  const int slot = slot_idx[j];
  if (slot <= 0 || slot >= c.num_slots) return;
  float *row = states + j * stride + ((int64_t)h * c.dv + rb * 16 + m) * DK + 4 * q;
  uint8_t *at = c.state + (int64_t)slot * c.state_stride + ((int64_t)h * nrb + rb) * (CH * 1024) + lane * 16;
  u32x4 ch[CH];
  if constexpr (READ) {
#pragma unroll
    for (int u = 0; u < CH; ++u) ch[u] = ld16(at + u * 1024);
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
      *reinterpret_cast<f32x4 *>(row + 16 * t) =
          f32x4{state_value<ST>(ch, 4 * t), state_value<ST>(ch, 4 * t + 1), state_value<ST>(ch, 4 * t + 2),
                state_value<ST>(ch, 4 * t + 3)};
  } else {
    float x[DK / 4];
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(row + 16 * t);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[4 * t + r] = v[r];
    }
    state_encode<ST, DK>(x, ch);
#pragma unroll
    for (int u = 0; u < CH; ++u) st16(at + u * 1024, ch[u]);
    // this row block's share of the rings: its columns of v, and from block 0
    // the gates and (a group's first head) k
    uint8_t *v = c.vc + (int64_t)slot * c.v_stride + ((int64_t)h * c.L * c.dv + rb * 16) * 2;
    for (int i = lane; i < c.L * 2; i += 64) st16(v + (int64_t)(i >> 1) * c.dv * 2 + (i & 1) * 16, u32x4{0, 0, 0, 0});
    if (rb == 0) {
      float2 *g = reinterpret_cast<float2 *>(c.gc + (int64_t)slot * c.g_stride) + (int64_t)h * c.L;
      for (int i = lane; i < c.L; i += 64) g[i] = float2{0.f, 0.f};
      if (h % c.hpg == 0) {
        uint8_t *k = c.kc + (int64_t)slot * c.k_stride + (int64_t)(h / c.hpg) * c.L * DK * 2;
        for (int i = lane; i < c.L * DK / 8; i += 64) st16(k + i * 16, u32x4{0, 0, 0, 0});
      }
      if (h == 0 && lane == 0) c.ring_start[slot] = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <int ST, int DK>
hipError_t delta_step_dk(const DCache &c, const DStep &s, int out_type, hipStream_t st) {
  constexpr int RB = kStepWaveChunks / dchunks(ST, DK);
  const int parts = (c.dv / 16 + RB - 1) / RB;
  const int64_t nwaves = (int64_t)s.batch * c.Hv * parts;
  const dim3 grid(xcd_grid(nwaves)), block(64);
  if (out_type == kOutF32) {
    if (c.L <= 16)
      delta_step_kernel<ST, kOutF32, 16, DK><<<grid, block, 0, st>>>(c, s, parts, nwaves);
    else
      delta_step_kernel<ST, kOutF32, 32, DK><<<grid, block, 0, st>>>(c, s, parts, nwaves);
  } else {
    if (c.L <= 16)
      delta_step_kernel<ST, kOutBF16, 16, DK><<<grid, block, 0, st>>>(c, s, parts, nwaves);
    else
      delta_step_kernel<ST, kOutBF16, 32, DK><<<grid, block, 0, st>>>(c, s, parts, nwaves);
  }
  return hipGetLastError();
}

template <int ST>
hipError_t delta_step_st(const DCache &c, const DStep &s, int out_type, hipStream_t st) {
  return c.dk == 64 ? delta_step_dk<ST, 64>(c, s, out_type, st) : delta_step_dk<ST, 128>(c, s, out_type, st);
}

template <int ST, int DK>
hipError_t delta_flush_dk(const DCache &c, const int32_t *slot_idx, const int32_t *num_fold, int n, hipStream_t st) {
  constexpr int RB = kStepWaveChunks / dchunks(ST, DK);
  const int parts = (c.dv / 16 + RB - 1) / RB;
  const int64_t nwaves = (int64_t)n * c.Hv * parts;
  const dim3 grid(xcd_grid(nwaves)), block(64);
  if (c.L <= 16)
    delta_flush_kernel<ST, 16, DK><<<grid, block, 0, st>>>(c, slot_idx, num_fold, parts, nwaves);
  else
    delta_flush_kernel<ST, 32, DK><<<grid, block, 0, st>>>(c, slot_idx, num_fold, parts, nwaves);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  delta_ring_advance_kernel<ST><<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st>>>(c, slot_idx, num_fold, n);
  return hipGetLastError();
}

template <int ST>
hipError_t delta_flush_st(const DCache &c, const int32_t *slot_idx, const int32_t *num_fold, int n, hipStream_t st) {
  return c.dk == 64 ? delta_flush_dk<ST, 64>(c, slot_idx, num_fold, n, st)
                    : delta_flush_dk<ST, 128>(c, slot_idx, num_fold, n, st);
}

template <int ST, bool READ>
hipError_t delta_state_st(const DCache &c, float *states, int64_t stride, const int32_t *slot_idx, int n,
                          hipStream_t st) {
  const int64_t nwaves = (int64_t)n * c.Hv * (c.dv / 16);
  if (c.dk == 64)
    delta_state_kernel<ST, 64, READ><<<dim3((unsigned)nwaves), dim3(64), 0, st>>>(c, states, stride, slot_idx, nwaves);
  else
    delta_state_kernel<ST, 128, READ><<<dim3((unsigned)nwaves), dim3(64), 0, st>>>(c, states, stride, slot_idx, nwaves);
  return hipGetLastError();
}

template <int ST>
hipError_t delta_init_st(const DCache &c, const float *states, int64_t stride, const int32_t *slot_idx, int n,
                         hipStream_t st) {
  return delta_state_st<ST, false>(c, const_cast<float *>(states), stride, slot_idx, n, st);
}

template <int ST>
hipError_t delta_read_st(const DCache &c, float *states, int64_t stride, const int32_t *slot_idx, int n,
                         hipStream_t st) {
  return delta_state_st<ST, true>(c, states, stride, slot_idx, n, st);
}

}  // namespace ssu
